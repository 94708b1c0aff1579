"""The gradient of a step's decay is made of what crosses that step alone."""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta
from test_gpu_delta import BF, F32, cuda, inputs

pytestmark = pytest.mark.gpu
SIZES = [(64, 64), (128, 64), (64, 128), (40, 24)]


def gradients(i, rest, dev):
    c, dy, h0, dend = cuda(i, dev), rest["dy"].to(dev), rest["h0"].to(dev), rest["dh_final"].to(dev)
    _, saved = lrs.delta_rule_fwd(**c, h0=h0, save="states")
    c.pop("v")
    return lrs.delta_rule_bwd(**c, dy=dy, saved=saved, dh_final=dend)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("cuts", [[10], [0, 31, 94], [63, 64, 65, 129], [1, 2, 40, 41, 120]])
def test_a_step_without_decay_left_has_no_gradient(cuda_device, dtype, K, V, cuts):
    """Nothing reaches across it: exactly 0, whatever the steps around it give."""
    i, rest = inputs(1, 1, 130, 1, 2, K, V, dtype)
    i["g"][:, cuts] = float("-inf")
    dg = gradients(i, rest, cuda_device)["dg"]
    assert torch.count_nonzero(dg[:, cuts]) == 0
    kept = [t for t in range(1, 129) if t not in cuts and t - 1 not in cuts]
    assert torch.count_nonzero(dg[:, kept]) == dg[:, kept].numel()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
def test_a_strong_decay_keeps_its_accuracy(cuda_device, dtype, K, V):
    """A decay of e^-60 leaves 1e-26 of what crosses its step: the gradient is that small, and right.

    The bound is that of test_gpu_delta.py (its largest error, relative to the value and to the 2-norm of the terms),
    of each of these steps by itself."""
    at = [7, 33, 70, 127]
    i, rest = inputs(2, 1, 140, 1, 2, K, V, dtype)
    i["g"][:, at] = -60.0
    got = gradients(i, rest, cuda_device)["dg"][0, at].double().cpu().numpy()
    want = delta.delta_rule_bwd(**i, dy=rest["dy"], h0=rest["h0"], dh_final=rest["dh_final"])
    value, terms = want["dg"][0, at], want["dg_terms"][0, at]
    assert np.all(np.abs(value) < 1e-20)
    bound = (1e-4 if dtype == F32 else 2e-2) * (np.abs(value) + terms)
    assert np.all(np.abs(got - value) <= bound), (got, value, bound)
