"""The root-mean-square norm on the GPU against the fp64 oracle.

Bounds: fp32 sums over a row, 1e-6 of the row's largest value (a tree of at
most 2^15 terms, 2^-24 each, the square root halves it); an output in bf16 adds
half a step, 2^-8 of the value; an 8-bit one half a step of its group's scale
(0.5 / 127 of the group's largest value, which is itself off by 1e-6).  dx is a difference,
r w dy - r (s r) mean(w dy s r): each term is within 1e-6 of its own size, but
they may cancel (in a row of one column they are equal), so the difference is
within 1e-6 of the larger term, |r| max|w dy| (1 + max|s r|^2), not of dx.
"""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta, gated

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (3, 7), (5, 64), (2, 65), (33, 128), (4, 200), (7, 1536), (3, 1537), (2, 2560), (1, 4096), (2, 9000),
         (2, 16384), (1, 32768), (1, 40000), (1300, 72), (1, 8), (700, 2048)]


def terms(dy, s, w, ds=None):
    """The size of the terms that dx is the sum of, by row."""
    s = gated.f64(s)
    r = 1 / np.sqrt((s ** 2).mean(-1, keepdims=True) + 1e-6)
    size = r * np.max(np.abs(gated.f64(dy) * gated.f64(w)), axis=-1, keepdims=True)
    size = size * (1 + np.max(np.abs(s * r), axis=-1, keepdims=True) ** 2)
    return size if ds is None else size + np.max(np.abs(gated.f64(ds)), axis=-1, keepdims=True)


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def close(got, want, scale=1e-6, top=None):
    """Within half a step of the type and `scale` of the row's largest value, or of `top`."""
    g = got.double().cpu().numpy()
    top = np.max(np.abs(want), axis=-1, keepdims=True) if top is None else top
    assert np.all(np.abs(g - want) <= HALF[got.dtype] * np.abs(want) + scale * top + 1e-30), np.max(np.abs(g - want))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_and_gradients(cuda_device, dtype, residual, rows, cols):
    dev = cuda_device
    x, r = (3 * rand(1, rows, cols)).to(dtype), rand(2, rows, cols).to(dtype) if residual else None
    w = 1 + 0.3 * rand(3, cols)
    dy, ds = rand(4, rows, cols).to(dtype), rand(5, rows, cols).to(dtype) if residual else None
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    got = lrs.rms_norm_fwd(on(x), on(w), residual=on(r), save=True)
    y, s, rstd = delta.rms_norm(x, w, r)
    close(got[0], y)
    close(got[-1][None], rstd[None])
    if residual:
        close(got[1], s)
    g = lrs.rms_norm_bwd(on(dy), on(x), on(w), got[-1], residual=on(r), ds=on(ds))
    dx, dw = delta.rms_norm_bwd(dy, s, w, ds)
    size = (np.abs(gated.f64(dy) * s) * rstd[:, None]).sum(0)
    close(g["dx"], dx, 1e-6, terms(dy, s, w, ds))
    assert np.all(np.abs(g["dweight"].double().cpu().numpy() - dw) <= 2e-6 * size)
    if residual:
        # at the sum as it was kept; the factor is the unrounded sum's: off by half a step at most
        g = lrs.rms_norm_bwd(on(dy), got[1], on(w), got[-1], ds=on(ds))
        dx, dw = delta.rms_norm_bwd(dy, got[1], w, ds)
        close(g["dx"], dx, 1e-6 + 3 * HALF[dtype], terms(dy, got[1], w, ds))
        assert np.all(np.abs(g["dweight"].double().cpu().numpy() - dw) <= (2e-6 + HALF[dtype]) * size)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_8bit_output(cuda_device, dtype, residual, rows, cols):
    x, r = (3 * rand(1, rows, cols)).to(dtype), rand(2, rows, cols).to(dtype) if residual else None
    w = 1 + 0.3 * rand(3, cols)
    got = lrs.rms_norm_fwd(x.to(cuda_device), w.to(cuda_device), residual=None if r is None else r.to(cuda_device),
                           out="8bit")
    y, s, _ = delta.rms_norm(x, w, r)
    back = lrs.ckpt8_load(got[0], got[1], F32).double().cpu().numpy()
    for c in range(0, cols, 64):
        top = np.max(np.abs(y[:, c:c + 64]), axis=-1, keepdims=True)
        row = np.max(np.abs(y), axis=-1, keepdims=True)
        # half a step, the value's own error, and the scale's
        assert np.all(np.abs(back[:, c:c + 64] - y[:, c:c + 64]) <= 0.5 / 127 * top + 3e-6 * row)
    # the same bits as the fp32 values kept in 8 bits
    if not residual and dtype == F32:
        q, scale = lrs.ckpt8_save(lrs.rms_norm_fwd(x.to(cuda_device), w.to(cuda_device)))
        assert torch.equal(q, got[0]) and torch.equal(scale, got[1])
    if residual:
        close(got[2], s)


def test_edges(cuda_device):
    zero = torch.zeros(3, 64, dtype=BF, device=cuda_device)
    assert torch.count_nonzero(lrs.rms_norm_fwd(zero)) == 0
    q, scale = lrs.rms_norm_fwd(zero, out="8bit")
    assert torch.count_nonzero(q) == 0 and torch.count_nonzero(scale) == 0
    # a row with a NaN, or an infinity, spoils no other
    x = rand(6, 4, 2048).to(cuda_device)
    want = lrs.rms_norm_fwd(x)
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y = lrs.rms_norm_fwd(x)
    assert torch.equal(y[[0, 3]], want[[0, 3]]) and torch.isnan(y[1]).all()
    back = lrs.ckpt8_load(*lrs.rms_norm_fwd(x, out="8bit"))
    assert torch.isfinite(back[[0, 3]].float()).all() and torch.isnan(back[1].float()).all()
    # any number of leading dimensions, no weight
    x = rand(7, 2, 3, 5, 64).to(cuda_device)
    assert torch.equal(lrs.rms_norm_fwd(x).view(-1, 64), lrs.rms_norm_fwd(x.view(-1, 64)))
    y, rstd = lrs.rms_norm_fwd(x, save=True)
    g = lrs.rms_norm_bwd(x, x, None, rstd)
    assert g["dweight"] is None and g["dx"].shape == x.shape


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cols", [64, 2048])
def test_rows_off_16_bytes(cuda_device, dtype, cols):
    room = torch.zeros(5 * cols + 1, dtype=dtype, device=cuda_device)
    room[1:] = rand(8, 5 * cols).to(cuda_device)
    x = room[1:].view(5, cols)
    w = 1 + 0.3 * rand(9, cols).to(cuda_device)
    y, rstd = lrs.rms_norm_fwd(x, w, save=True)
    close(y, delta.rms_norm(x, w)[0])
    g = lrs.rms_norm_bwd(x, x, w, rstd)
    dx, dw = delta.rms_norm_bwd(x, x, w)
    close(g["dx"], dx, 3e-6, terms(x, x, w))
    assert np.allclose(g["dweight"].double().cpu().numpy(), dw, rtol=1e-5, atol=1e-4)


def test_same_bits_on_another_stream_and_in_a_graph(cuda_device):
    x, r = rand(10, 1000, 2560).to(BF).to(cuda_device), rand(11, 1000, 2560).to(BF).to(cuda_device)
    w = 1 + 0.3 * rand(12, 2560).to(cuda_device)

    def both():
        y, s, rstd = lrs.rms_norm_fwd(x, w, residual=r, save=True)
        q, scale, _ = lrs.rms_norm_fwd(x, w, residual=r, out="8bit")
        g = lrs.rms_norm_bwd(y, s, w, rstd, ds=x)
        return y, s, rstd, q, scale, g["dx"], g["dweight"]

    first = [t.clone() for t in both()]
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = both()
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    for t in third:
        t.fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals_of_the_binding(cuda_device):
    x, w = rand(13, 4, 64).to(cuda_device), rand(14, 64).to(cuda_device)
    for args, kw in (((x[:, ::2],), {}), ((x.half(),), {}), ((x, w[:5]), {}), ((x, w.to(BF)), {}),
                     ((x, w), dict(residual=x[:2])), ((x, w), dict(residual=x.to(BF))), ((x, w), dict(out="16bit")),
                     ((x, w), dict(eps=-1.0)), ((x[:0], w), {}), ((x, w), dict(residual=3))):
        with pytest.raises((TypeError, ValueError, lrs.SsmError)):
            lrs.rms_norm_fwd(*args, **kw)
    y, rstd = lrs.rms_norm_fwd(x, w, save=True)
    for args, kw in (((y, x[:2], w, rstd), {}), ((y, x, w, rstd[:3]), {}), ((y, x, w, None), {}),
                     ((y, x.to(BF), w, rstd), {}), ((y, x, w, rstd), dict(ds=x[:1])), ((y, None, w, rstd), {})):
        with pytest.raises((TypeError, ValueError, lrs.SsmError)):
            lrs.rms_norm_bwd(*args, **kw)
