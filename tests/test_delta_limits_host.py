"""Sizes that the gated delta rule does not take are refused as such, also by a
caller that was told to bring no scratch for them (CPU only)."""
import pytest

import linear_recurrence_ssm_gb300 as lrs
from test_delta_host import INVALID, UNSUPPORTED, bwd, fwd, swapped


@pytest.mark.parametrize("call,pointers", [(fwd, 12), (bwd, 16)])
def test_sizes_without_scratch(call, pointers):
    no_scratch = swapped(pointers, pointers - 1, None)
    for kw in (dict(K=257), dict(V=300), dict(L=2 ** 31 - 1)):
        assert call(no_scratch, **kw) == UNSUPPORTED, kw
    for kw in (dict(), dict(K=0), dict(G=3)):
        assert call(no_scratch, **kw) == INVALID, kw
    for size in (lrs.library().delta_rule_fwd_scratch, lrs.library().delta_rule_bwd_scratch):
        assert size(1, 8, 2, 4, 257, 8, 1, 1) == 0
