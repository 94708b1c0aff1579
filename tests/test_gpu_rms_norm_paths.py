"""Every path of the norm's kernels on the GPU against the fp64 oracle: widths of
two and four vectors a thread, so many rows that each thread block takes several
turns, and outputs that lie where an input lay.

Bounds of y, s and dx as in test_gpu_rms_norm.py.  dweight is a sum over rows of
dy s r: each term is off by 1e-6 of its size (s r), and a partial sum is rounded
at every addition.  A column's sum goes through at most 33 additions a thread
(40000 rows over 1216 parts; 22 in the vector kernels, whose 304 blocks at least
run at a time), 3 and 8 that join the lanes and the warps of a block, and, of at
most 1216 parts, 10 a thread, 2 and 5: less than 64 in a row, 2^-24 each of what is
summed: 1e-6 + 64 2^-24 = 4.9e-6 of the terms' sum.
"""
import ctypes

import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta, gated
from test_gpu_rms_norm import BF, F32, HALF, close, rand, terms

pytestmark = pytest.mark.gpu
WIDE = [(3, 4104), (2, 6000), (5, 8192), (1500, 8192)]                      # two vectors a thread
TURNS = [(5000, 2048), (3000, 2560), (100001, 64), (50003, 136), (20000, 256)]
OTHER = [(3, 8200), (2, 12288), (3000, 1537), (40000, 33)]                  # single elements


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", WIDE + TURNS + OTHER)
def test_gradients(cuda_device, dtype, residual, rows, cols):
    dev = cuda_device
    x, r = (3 * rand(1, rows, cols)).to(dtype), rand(2, rows, cols).to(dtype) if residual else None
    w = 1 + 0.3 * rand(3, cols)
    dy, ds = rand(4, rows, cols).to(dtype), rand(5, rows, cols).to(dtype) if residual else None
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    got = lrs.rms_norm_fwd(on(x), on(w), residual=on(r), save=True)
    y, s, rstd = delta.rms_norm(x, w, r)
    close(got[0], y)
    close(got[-1][None], rstd[None])
    size = (np.abs(gated.f64(dy) * s) * rstd[:, None]).sum(0)
    kept = got[-1]
    if residual:
        close(got[1], s)
    for more in (ds, None):
        g = lrs.rms_norm_bwd(on(dy), on(x), on(w), kept, residual=on(r), ds=on(more))
        dx, dw = delta.rms_norm_bwd(dy, s, w, more)
        close(g["dx"], dx, 1e-6, terms(dy, s, w, more))
        assert np.all(np.abs(g["dweight"].double().cpu().numpy() - dw) <= 4.9e-6 * size)
        # dx alone is the same
        alone = lrs.rms_norm_bwd(on(dy), on(x), on(w), kept, residual=on(r), ds=on(more), need_dweight=False)
        assert alone["dweight"] is None and torch.equal(alone["dx"], g["dx"])


def at(t):
    return None if t is None else t.data_ptr()


def norm(x, r, w, s, y=None, q=None, scale=None, rstd=None):
    return lrs.library().rms_norm_fwd(at(x), at(r), at(w), 1e-6, at(s), at(y), at(q), at(scale), at(rstd), *x.shape,
                                      int(x.dtype is BF), torch.cuda.current_stream().cuda_stream)


IN_PLACE = [(70, 64), (40, 256), (9, 1536), (5, 2048), (3, 8192), (2, 32768), (5, 33), (3, 1537), (2, 40000)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,cols", IN_PLACE)
def test_the_sum_in_an_input_s_place(cuda_device, dtype, rows, cols):
    x, r = (rand(n, rows, cols).to(dtype).to(cuda_device) for n in (1, 2))
    w = (1 + 0.3 * rand(3, cols)).to(cuda_device)
    y, s, rstd = lrs.rms_norm_fwd(x, w, residual=r, save=True)
    q, scale, _ = lrs.rms_norm_fwd(x, w, residual=r, out="8bit")
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
        assert norm(a, b, w, (a, b)[which], y=y2, rstd=rstd2) == 0
        assert torch.equal((a, b)[which], s) and torch.equal((b, a)[which], (r, x)[which])
        assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
        a, b = x.clone(), r.clone()
        q2, scale2 = torch.empty_like(q), torch.empty_like(scale)
        assert norm(a, b, w, (a, b)[which], q=q2, scale=scale2) == 0
        assert torch.equal((a, b)[which], s) and torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", IN_PLACE)
def test_dx_in_the_sum_s_gradient_s_place(cuda_device, dtype, residual, rows, cols):
    x, r, dy, ds = (rand(n, rows, cols).to(dtype).to(cuda_device) for n in (1, 2, 3, 4))
    r = r if residual else None
    w = (1 + 0.3 * rand(5, cols)).to(cuda_device)
    rstd = lrs.rms_norm_fwd(x, w, residual=r, save=True)[-1]
    want = lrs.rms_norm_bwd(dy, x, w, rstd, residual=r, ds=ds)
    dw = torch.empty_like(want["dweight"])
    scratch = torch.empty(min(rows, 1216) * cols, device=cuda_device)
    assert lrs.library().rms_norm_bwd(at(dy), at(x), at(r), at(w), at(rstd), at(ds), at(ds), at(dw), at(scratch), rows,
                                      cols, int(dtype is BF), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert torch.equal(ds, want["dx"]) and torch.equal(dw, want["dweight"])
