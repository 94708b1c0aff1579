"""Refusals of the gated delta rule that only a call on CUDA tensors reaches."""
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from test_gpu_delta import BF

pytestmark = pytest.mark.gpu
INVALID, UNSUPPORTED = 1, 2


def calls(K, V, dev):
    z = lambda *shape: torch.zeros(*shape, dtype=BF, device=dev)  # noqa: E731
    q, v, g = z(1, 70, 1, K), z(1, 70, 1, V), z(1, 70, 1)
    saved = dict(states=z(2, 1, V, K), errors=z(1, 70, 1, V))
    yield lambda: lrs.delta_rule_fwd(q, q, v, g, g)
    yield lambda: lrs.delta_rule_bwd(q, q, g, g, v, saved)
    yield lambda: lrs.delta_rule_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0],
                                      torch.zeros(1, 1, V, K, device=dev))


@pytest.mark.parametrize("K,V,status", [(264, 64, UNSUPPORTED), (64, 257, UNSUPPORTED), (0, 64, INVALID), (64, 0, INVALID)])
def test_head_sizes(cuda_device, K, V, status):
    for call in calls(K, V, cuda_device):
        with pytest.raises(lrs.SsmError) as e:
            call()
        assert e.value.status == status
