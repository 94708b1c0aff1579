"""Gradients of the gated delta rule, and the norm's, where offsets pass 32 bits;
head sizes at the ends of what each path takes."""
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from test_gpu_delta import BF, F32, check, close, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,G", [(BF, 32), (BF, 2), (F32, 2)])
def test_gradients_of_tokens_beyond_32_bits(cuda_device, dtype, G):
    """More than 2^31 elements in v and its gradient; decays of e^-0.5 and less a step, so that the first and the last
    256 steps are those of calls of 640 steps (e^-192 of what lies beyond is left)."""
    L, H, D, tail = 64 * 8210, 32, 128, 640
    g = torch.Generator(device=cuda_device).manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=cuda_device, dtype=dtype)

    q, k = rand(1, L, G, D).div_(11.3), rand(1, L, G, D).div_(11.3)
    v, dy = rand(1, L, H, D), rand(1, L, H, D)
    gate = (-torch.rand(1, L, H, generator=g, device=cuda_device) - 0.5).to(dtype)
    beta = torch.rand(1, L, H, generator=g, device=cuda_device).to(dtype)
    dend = torch.randn(1, H, D, D, generator=g, device=cuda_device)
    assert v.numel() > 2 ** 31

    def grads(a, b, dend):
        w = [t[:, a:b].contiguous() for t in (q, k, v, gate, beta)]
        _, saved = lrs.delta_rule_fwd(*w, save="states")
        return lrs.delta_rule_bwd(*w[:2], *w[3:], dy[:, a:b].contiguous(), saved, dh_final=dend)

    whole = grads(0, L, dend)
    first, last = grads(0, tail, None), grads(L - tail, L, dend)
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        close(whole[name][:, :256], first[name][:, :256].double().cpu().numpy(), dtype, name)
        close(whole[name][:, -256:], last[name][:, -256:].double().cpu().numpy(), dtype, name)
    close(whole["dh0"], first["dh0"].double().cpu().numpy(), F32, "dh0")
    lrs.ssm_check_device_errors()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1050000, 2048), (1050000, 2049), (34000000, 64)])
def test_norm_of_rows_beyond_32_bits(cuda_device, dtype, rows, cols):
    """Rows are independent of one another: the last ones are those of a call of their own."""
    g = torch.Generator(device=cuda_device).manual_seed(2)
    x, dy = (torch.randn(rows, cols, generator=g, device=cuda_device, dtype=dtype) for _ in range(2))
    w = 1 + 0.3 * torch.randn(cols, generator=g, device=cuda_device)
    assert x.numel() > 2 ** 31
    y, s, rstd = lrs.rms_norm_fwd(x, w, residual=dy, save=True)
    few = lrs.rms_norm_fwd(x[-50:].contiguous(), w, residual=dy[-50:].contiguous(), save=True)
    assert all(torch.equal(a[-50:], b) for a, b in zip((y, s, rstd), few))
    q, scale = lrs.rms_norm_fwd(s, w, out="8bit")
    few = lrs.rms_norm_fwd(s[-50:].contiguous(), w, out="8bit")
    assert torch.equal(q[-50:], few[0]) and torch.equal(scale[:, -50:], few[1])
    del y, q, scale
    got = lrs.rms_norm_bwd(dy, s, w, rstd, ds=x)
    few = lrs.rms_norm_bwd(dy[-50:].contiguous(), s[-50:].contiguous(), w, rstd[-50:].contiguous(), ds=x[-50:].contiguous())
    assert torch.equal(got["dx"][-50:], few["dx"])
    # dweight: a thread adds at most 34000000 / (304 x 64) pairs of rows, less than 3600 additions with those that join
    # the threads (see test_gpu_rms_norm_paths.py).  Each rounds its partial sum by 2^-24 at most, and terms whose signs
    # are as good as drawn keep a thread's partial sums below four times their 2-norm; threads are independent of one
    # another, so that their 2-norms and errors add up by squares: 4 x 3600 2^-24 of the 2-norm of all terms
    want, norm = torch.zeros(cols, dtype=torch.float64, device=cuda_device), 0.0
    for a in range(0, rows, 50000):
        t = dy[a:a + 50000].double() * (s[a:a + 50000].double() * rstd[a:a + 50000, None].double())
        want += t.sum(0)
        norm = norm + t.square().sum(0)
    bound = 4 * 3600 * 2.0 ** -24 * norm.sqrt()
    assert torch.all((got["dweight"].double() - want).abs() <= bound)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(8, 8), (8, 128), (128, 8), (104, 56), (64, 256), (128, 200), (256, 64), (129, 65), (136, 64)])
def test_head_sizes(cuda_device, dtype, K, V):
    i, rest = inputs(K + V, 1, 150, 1, 2, K, V, dtype, n=2)
    check(i, rest, cuda_device, [0, 70, 150])
