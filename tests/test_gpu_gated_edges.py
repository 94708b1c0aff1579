"""GPU tests of the gated linear recurrence at its edges: many sequences,
infinities and NaN where a reset drops them, rates beyond fp32."""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import gated

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- lam's gradient over many sequences -----------------------------------------------
def _dlam(one, Bs, lam, h0, dev):
    """dlam of Bs copies of one sequence (x, gate_r, gate_i, dy), and of the
    oracle: Bs times that of one, with the size of its terms."""
    L, ED = one[0].shape[1:]
    x, r, i, dy = (t.expand(Bs, L, ED).contiguous().to(dev) for t in one)
    d = (x, r, i, lam.to(dev))
    _, saved = lrs.gated_scan_fwd(*d, h0=h0.expand(Bs, ED).contiguous().to(dev), save="states")
    g = lrs.gated_scan_bwd(*d, dy, saved)
    again = lrs.gated_scan_bwd(*d, dy, saved)
    assert all(torch.equal(g[k], again[k]) for k in g)
    ref = gated.gated_scan_bwd(*one[:3], lam, one[3], saved["states"][:1])
    return g["dlam"].double().cpu().numpy(), Bs * ref["dlam"], Bs * ref["size_lam"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,L,ED", [(30000, 1, 64), (65535, 1, 33), (5000, 7, 65), (1024, 128, 40)])
def test_dlam_of_many_like_sequences(cuda_device, Bs, L, ED, dtype):
    """Like sequences give like terms, whose sum rounds the same way at every
    addition: a single running sum in fp32 loses up to Bs 2^-26 of it, 4e-4
    for 30000.  Each term is off by 2 (16 + L) 2^-21 of its size as in the
    other tests (a gradient joins two scans), and their sum by no more, per
    channel."""
    gen = torch.Generator().manual_seed(Bs + ED)
    one = [torch.randn(1, L, ED, generator=gen).to(TYPES[dtype]) for _ in range(4)]
    lam, h0 = torch.randn(ED, generator=gen) - 4.0, torch.randn(1, ED, generator=gen)
    got, want, size = _dlam(one, Bs, lam, h0, cuda_device)
    assert (np.abs(got - want) <= 2 * (16 + L) * 2.0 ** -21 * size).all(), np.max(np.abs(got - want) / size)


def test_dlam_of_infinite_and_nan_terms(cuda_device):
    """An infinite term makes an infinite sum, a NaN a NaN, in its channel alone."""
    gen = torch.Generator().manual_seed(3)
    x, r, i, dy = (torch.randn(40, 3, 64, generator=gen) for _ in range(4))
    dy[7, 1, 5], dy[9, 2, 40] = float("inf"), float("nan")
    d = [t.to(cuda_device) for t in (x, r, i, torch.full((64,), -4.0))]
    _, saved = lrs.gated_scan_fwd(*d, save="states")
    dlam = lrs.gated_scan_bwd(*d, dy.to(cuda_device), saved)["dlam"].cpu()
    assert torch.isinf(dlam[5]) and torch.isnan(dlam[40])
    dlam[5] = dlam[40] = 0
    assert torch.isfinite(dlam).all()


# ---- infinities and NaN next to a reset -------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ED,e", [(128, 1), (130, 32)])
@pytest.mark.parametrize("at", [3, 20, 100])
@pytest.mark.parametrize("nan", [float("nan"), -float("nan")])
def test_nan_gate_behind_a_reset(cuda_device, ED, e, at, nan, dtype):
    """A NaN gate of channel 0 soon after a reset, in the same 8 steps, is
    channel 0's alone: channel `e` (the one that a lane takes together with it)
    still drops the infinite state before the reset and, in the gradients, the
    infinite adjoint behind it.  Bounds as in test_gpu_gated."""
    L = 300
    gen = torch.Generator().manual_seed(at + ED)
    x, r, i, dy = (torch.randn(1, L, ED, generator=gen).to(TYPES[dtype]) for _ in range(4))
    lam = torch.full((ED,), -4.0)
    reset = torch.zeros(1, L, dtype=torch.uint8)
    reset[0, at] = 1
    r[0, at + 1, 0] = nan
    others = [k for k in range(ED) if k != 0]
    dev = [t.to(cuda_device) for t in (r, i, lam, reset)]

    bad = x.clone()
    bad[0, at - 1, e] = float("inf")
    y, hf, saved = lrs.gated_scan_fwd(bad.to(cuda_device), *dev[:3], reset=dev[3], return_final_state=True,
                                      save="states")
    ref = gated.gated_scan(x, r, i, lam, reset=reset)
    bound = (16 + L) * 2.0 ** -21 * max(1.0, float(np.max(np.abs(ref[:, :, others]))))
    got = y.double().cpu().numpy()[0, at:][:, others]
    want = ref[0, at:][:, others]
    assert (np.abs(got - want) <= bound + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)).all()
    assert (np.abs(hf.double().cpu().numpy() - ref[:, -1])[:, others] <= bound).all()
    assert torch.isnan(y[0, at + 1:, 0]).all()

    dy[0, at + 1, e] = float("inf")
    x = x.to(cuda_device)
    _, saved = lrs.gated_scan_fwd(x, *dev[:3], reset=dev[3], save="states")
    g = lrs.gated_scan_bwd(x, *dev[:3], dy.to(cuda_device), saved, reset=dev[3])
    for k in ("dx", "dgate_r", "dgate_i"):
        assert torch.isfinite(g[k][0, :at]).all(), k
    assert torch.isfinite(g["dh0"]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_gate_without_a_reset(cuda_device, dtype):
    """A NaN gate (of either sign) or rate of one channel leaves the others
    alone, also where resets are given, over a cluster's blocks, too."""
    L, ED = 1500, 128
    gen = torch.Generator().manual_seed(7)
    x, r, i, dy = (torch.randn(1, L, ED, generator=gen).to(TYPES[dtype]) for _ in range(4))
    lam = torch.full((ED,), -4.0)
    reset = torch.zeros(1, L, dtype=torch.uint8)
    reset[0, 3] = 1
    want = [t.to(cuda_device) for t in (x, r, i, lam)]
    reset = reset.to(cuda_device)
    r[0, 700, 0], r[0, 900, 2], lam[4] = float("nan"), -float("nan"), -float("nan")
    got = [t.to(cuda_device) for t in (x, r, i, lam)]
    dy = dy.to(cuda_device)
    others = [k for k in range(ED) if k not in (0, 2, 4)]

    def both(inp):
        y, hf, saved = lrs.gated_scan_fwd(*inp, reset=reset, return_final_state=True, save="states")
        g = lrs.gated_scan_bwd(*inp, dy, saved, reset=reset)
        return [t[..., others].float() for t in (y, hf, saved["states"], *g.values())]

    # a NaN rate sends its warp through the general form of the decay: up to
    # rounding, (16 + L) 2^-21 of the largest value and a neighbouring bf16
    for a, b in zip(both(got), both(want)):
        bound = 2 * (16 + L) * 2.0 ** -21 * max(1.0, b.abs().max().item())
        assert ((a - b).abs() <= bound + (2.0 ** -7 * b.abs() if dtype == "bf16" else 0)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [float("nan"), float("inf"), -float("inf")])
def test_gate_of_a_reset_step_is_not_used(cuda_device, gate, dtype):
    """A reset step's decay is the constant 0: whatever its gate_r holds, y and
    the gradients are what they are with another gate, and its own is 0."""
    Bs, L, ED = 2, 150, 72
    gen = torch.Generator().manual_seed(11)
    x, r, i, dy = (torch.randn(Bs, L, ED, generator=gen).to(TYPES[dtype]).to(cuda_device) for _ in range(4))
    lam = torch.full((ED,), -4.0, device=cuda_device)
    reset = torch.zeros(Bs, L, dtype=torch.uint8, device=cuda_device)
    reset[0, 17] = reset[1, 0] = reset[1, 149] = 1

    def both(r):
        y, hf, saved = lrs.gated_scan_fwd(x, r, i, lam, reset=reset, return_final_state=True, save="states")
        return y, hf, lrs.gated_scan_bwd(x, r, i, lam, dy, saved, reset=reset)

    y, hf, g = both(r)
    odd = r.clone()
    odd[reset != 0] = gate
    y2, hf2, g2 = both(odd)
    assert torch.equal(y, y2) and torch.equal(hf, hf2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    assert not g2["dgate_r"][reset != 0].any()


# ---- rates beyond fp32 ------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lam,c", [(2e37, 8.0), (1e38, 8.0), (3e38, 8.0), (float("inf"), 8.0), (30.0, 3e37),
                                   (1.0, 3e38)])
def test_rates_beyond_fp32(cuda_device, lam, c, dtype):
    """c softplus(lam) above the largest fp32 is a decay of 0 where the gate is
    open, of 1 where it is shut: no NaN, in the scan, its gradients and the
    step.  A shut gate (-200) has s_r = 0 in fp32, e^-200 in the oracle: la is
    0 and -1e-48."""
    Bs, L, ED = 1, 70, 64
    gen = torch.Generator().manual_seed(5)
    x, r, i, dy = (torch.randn(Bs, L, ED, generator=gen).to(TYPES[dtype]) for _ in range(4))
    r[0, 5] = r[0, 40] = r[0, 69] = -200.0
    h0, dh = torch.randn(Bs, ED, generator=gen), torch.randn(Bs, ED, generator=gen)
    d = [t.to(cuda_device) for t in (x, r, i, torch.full((ED,), lam))]
    y, saved = lrs.gated_scan_fwd(*d, c=c, h0=h0.to(cuda_device), save="states")
    g = lrs.gated_scan_bwd(*d, dy.to(cuda_device), saved, c=c, dh_final=dh.to(cuda_device))
    big = torch.full((ED,), min(lam, 3e38))
    ref = gated.gated_scan(x, r, i, big, c, h0=h0)
    want = gated.gated_scan_bwd(x, r, i, big, dy, saved["states"], c, dh_final=dh)

    def near(got, ref, what):      # as in test_gpu_gated
        bound = 2 * (16 + L) * 2.0 ** -21 * max(1.0, float(np.max(np.abs(ref))))
        bound = bound + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0)
        assert (np.abs(got.double().cpu().numpy() - ref) <= bound).all(), what

    near(y, ref, "y")
    for k in g:
        near(g[k], want[k], k)
    states = h0.to(cuda_device)
    near(lrs.gated_scan_step(*[t[:, 0].contiguous() for t in d[:3]], d[3], states, c=c), ref[:, 0], "step")
    near(states, ref[:, 0], "state")


def test_a_nan_rate_stays(cuda_device):
    x = torch.randn(1, 40, 64, device=cuda_device)
    lam = torch.zeros(64, device=cuda_device)
    lam[7] = float("nan")
    y = lrs.gated_scan_fwd(x, x, x, lam)
    assert torch.isnan(y[..., 7]).all() and torch.isfinite(y[..., :7]).all() and torch.isfinite(y[..., 8:]).all()


# ---- waits that run out -----------------------------------------------------------------
@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("copy", [0, 1])
def test_waits_give_up(cuda_device, backward, copy):
    """A wait that cannot end gives up after its 20 ms, the hundred turns after
    it wait no more (they would take 2 s), 20 ms more pass for copies under
    way; the unit's error word is reported once, and the next calls are right."""
    lib, stream = lrs.library(), torch.cuda.current_stream(cuda_device)
    assert lib.ssm_check_device_errors(stream.cuda_stream) == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    assert lib.gated_selftest_wait_timeout(backward, copy, stream.cuda_stream) == 0
    end.record()
    assert lib.ssm_check_device_errors(stream.cuda_stream) == 5      # SSM_ERR_DEVICE_TIMEOUT
    assert lib.ssm_check_device_errors(stream.cuda_stream) == 0      # cleared
    assert 39.0 < start.elapsed_time(end) < 1000.0
    gen = torch.Generator().manual_seed(1)
    x, r, i = (torch.randn(1, 700, 64, generator=gen) for _ in range(3))
    lam = torch.full((64,), -4.0)
    d = [t.to(cuda_device) for t in (x, r, i, lam)]
    y, saved = lrs.gated_scan_fwd(*d, save="states")
    ref = gated.gated_scan(x, r, i, lam)
    bound = (16 + 700) * 2.0 ** -21 * max(1.0, float(np.max(np.abs(ref))))
    assert (np.abs(y.double().cpu().numpy() - ref) <= bound).all()
    g = lrs.gated_scan_bwd(*d, d[0], saved)
    want = gated.gated_scan_bwd(x, r, i, lam, x, saved["states"])
    bound = 2 * (16 + 700) * 2.0 ** -21 * max(1.0, float(np.max(np.abs(want["dx"]))))
    assert (np.abs(g["dx"].double().cpu().numpy() - want["dx"]) <= bound).all()
    assert lib.ssm_check_device_errors(stream.cuda_stream) == 0


# ---- the slowest decays -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("lam", [-50.0, -65.0, -70.0])
def test_slowest_decays(cuda_device, lam, fast, dtype):
    """m = sqrt(1 - a^2) to full relative accuracy as a -> 1: from h0 = 0, y is
    m's size (1e-11 to 1e-15), and within the usual bound of that, as are the
    gradients.  `fast` puts fast decays beside them, which are computed in
    another form."""
    Bs, L, ED = 1, 70, 64
    gen = torch.Generator().manual_seed(9)
    x, r, i, dy = (torch.randn(Bs, L, ED, generator=gen).to(TYPES[dtype]) for _ in range(4))
    lams = torch.full((ED,), lam)
    if fast:
        lams[1::2] = 1.0
    d = [t.to(cuda_device) for t in (x, r, i, lams)]
    y, saved = lrs.gated_scan_fwd(*d, save="states")
    g = lrs.gated_scan_bwd(*d, dy.to(cuda_device), saved)
    step = lrs.gated_scan_step(*[t[:, 0].contiguous() for t in d[:3]], d[3], torch.zeros(Bs, ED, device=cuda_device))
    ref = gated.gated_scan(x, r, i, lams)
    want = gated.gated_scan_bwd(x, r, i, lams, dy, saved["states"])
    slow = slice(0, ED, 2 if fast else 1)

    def near(got, ref, size, what):
        got = got.double().cpu().numpy()[..., slow]
        bound = 2 * (16 + L) * 2.0 ** -21 * np.max(np.abs(size[..., slow]))
        bound = bound + (2.0 ** -8 * np.abs(ref[..., slow]) if dtype == "bf16" else 0.0)
        assert (np.abs(got - ref[..., slow]) <= bound).all(), (what, np.max(np.abs(got - ref[..., slow])), np.max(bound))

    near(y, ref, ref, "y")
    near(step, ref[:, 0], ref[:, 0], "step")
    for k, size in (("dx", "dx"), ("dgate_i", "dgate_i"), ("dgate_r", "size"), ("dlam", "size_lam"), ("dh0", "dh0")):
        near(g[k], want[k], want[size], k)
