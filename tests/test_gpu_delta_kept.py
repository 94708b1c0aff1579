"""What the gated delta rule keeps for its gradients is written whole: places
of blocks that no sequence has, and rows that none covers, are 0."""
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from delta_calls import Guarded, forward
from test_gpu_delta import BF, F32, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (40, 24), (5, 3)])
@pytest.mark.parametrize("L,offsets", [(262, [0, 5, 5, 133, 262]), (262, [3, 67, 68, 200, 200]), (70, [0, 0, 0]),
                                       (262, [64, 65, 66, 262]), (2100, [100, 612, 612, 2000])])
def test_states_and_errors_are_written_whole(cuda_device, dtype, K, V, L, offsets):
    i, rest = inputs(1, 1, L, 1, 2, K, V, dtype, n=len(offsets) - 1)
    c, h0 = cuda(i, cuda_device), rest["h0"].to(cuda_device)
    o = torch.tensor(offsets, dtype=torch.int32, device=cuda_device)
    room = Guarded(cuda_device)
    status, out = forward(c, o, h0, room=room)
    assert status == 0 and room.untouched()
    used = torch.zeros(len(out["states"]), dtype=torch.bool)
    for n, (a, b) in enumerate(zip(offsets, offsets[1:])):
        used[a // 64 + n:a // 64 + n + -(-(b - a) // 64)] = True
    for w in out.values():
        assert torch.isfinite(w).all()
    assert torch.count_nonzero(out["states"][~used.to(cuda_device)]) == 0
    assert torch.count_nonzero(out["errors"][:, :offsets[0]]) == 0
    assert torch.count_nonzero(out["errors"][:, offsets[-1]:]) == 0
    y, hf, saved = lrs.delta_rule_fwd(**c, scale=1.0, offsets=o, h0=h0, return_final_state=True, save="states")
    assert torch.equal(y, out["y"]) and torch.equal(hf, out["h_final"])
    assert torch.equal(saved["errors"], out["errors"]) and torch.equal(saved["states"], out["states"])
