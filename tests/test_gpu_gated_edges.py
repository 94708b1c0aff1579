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
