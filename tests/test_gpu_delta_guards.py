"""No output or scratch of the gated delta rule is written outside its size, and
nothing of what lies in rows that no sequence covers enters a result."""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from delta_calls import Guarded, at, backward, forward, stream
from oracle import delta
from test_gpu_delta import BF, F32, close, cuda, inputs

pytestmark = pytest.mark.gpu
SIZES = [(64, 64), (128, 128), (72, 136), (40, 24), (5, 3)]


def both(i, rest, o, dev):
    room = Guarded(dev)
    c = {n: room.empty(*w.shape, dtype=w.dtype).copy_(w) for n, w in i.items()}      # reads before or behind: NaN or worse
    h0, dend = (rest[n].to(dev) for n in ("h0", "dh_final"))
    status, out = forward(c, o, h0, scale=0.3, room=room)
    assert status == 0
    dy = room.empty(*rest["dy"].shape, dtype=rest["dy"].dtype).copy_(rest["dy"])
    status, grads = backward(c, dy, out, o, dend, scale=0.3, room=room)
    assert status == 0
    torch.cuda.synchronize()
    assert room.untouched()
    lrs.ssm_check_device_errors()
    return out, grads


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("Bs,L,G,H,offsets", [(2, 65, 1, 2, None), (1, 1, 2, 2, None), (1, 262, 2, 2, [3, 67, 68, 200, 200]),
                                              (1, 1600, 1, 2, None), (1, 2100, 1, 1, [0, 0, 1900, 2000]), (1, 70, 1, 3, [0, 0, 0])])
def test_sizes(cuda_device, dtype, K, V, Bs, L, G, H, offsets):
    n = None if offsets is None else len(offsets) - 1
    i, rest = inputs(1, Bs, L, G, H, K, V, dtype, n=n)
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=cuda_device)
    out, grads = both(i, rest, o, cuda_device)
    for w in (*out.values(), *grads.values()):
        assert torch.isfinite(w).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("L,offsets", [(90, [5, 3, 300, 2, 90]), (90, [-7, 40, 10 ** 9, 10 ** 9, 2 ** 31 - 1]),
                                       (90, [90, 60, 30, 10, 0]), (90, [-1, -1, -1, -1, -1]), (2500, [0, 2400, 100, 2000, 10 ** 9]),
                                       (2500, [-5, 2500, 0, 2500, 0]), (2500, [2000, 1500, 1000, 500, 0])])
def test_bad_offsets(cuda_device, dtype, K, V, L, offsets):
    i, rest = inputs(2, 1, L, 1, 2, K, V, dtype, n=len(offsets) - 1)
    both(i, rest, torch.tensor(offsets, dtype=torch.int32, device=cuda_device), cuda_device)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("pages", [None, [3, -1, 0, 7, 2 ** 31 - 1], [-2 ** 31, 6, 5, 1, 2]])
def test_token_steps(cuda_device, dtype, K, V, pages):
    i, _ = inputs(3, 5, 1, 1, 2, K, V, dtype)
    room = Guarded(cuda_device)
    c = {n: room.empty(*w[:, 0].shape, dtype=w.dtype).copy_(w[:, 0]) for n, w in i.items()}
    y, pool = room.empty(5, 2, V, dtype=dtype), room.empty(7, 2, V, K, dtype=F32)
    before = torch.randn(7, 2, V, K, generator=torch.Generator().manual_seed(4))
    pool.copy_(before)
    p = None if pages is None else torch.tensor(pages, dtype=torch.int32, device=cuda_device)
    assert lrs.library().delta_rule_step(*(at(c[w]) for w in ("q", "k", "v", "g", "beta")), K ** -0.5, at(pool), at(p), at(y),
                                         5, 1, 2, K, V, 7, int(dtype is BF), stream()) == 0
    torch.cuda.synchronize()
    assert room.untouched()
    want, after = delta.delta_rule_step(**{n: w[:, 0] for n, w in i.items()}, states=before, pages=pages)
    close(y, want)
    close(pool, after)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("L,offsets", [(262, [3, 67, 68, 200, 200]), (2100, [100, 612, 612, 2000]), (70, [30, 30, 31]), (70, [9, 9, 9])])
def test_rows_that_no_sequence_covers(cuda_device, dtype, K, V, L, offsets):
    """A padded batch: NaN before the first sequence and behind the last, in every input."""
    i, rest = inputs(4, 1, L, 1, 2, K, V, dtype, n=len(offsets) - 1)
    o = torch.tensor(offsets, dtype=torch.int32, device=cuda_device)
    out, grads = both(i, rest, o, cuda_device)
    padded = [torch.cat((torch.full_like(w[:, :offsets[0]], float("nan")), w[:, offsets[0]:offsets[-1]],
                         torch.full_like(w[:, offsets[-1]:], float("nan"))), 1) for w in (*i.values(), rest["dy"])]
    out2, grads2 = both(dict(zip(i, padded)), dict(rest, dy=padded[-1]), o, cuda_device)
    for a, b in ((out, out2), (grads, grads2)):
        for name in a:
            assert torch.equal(a[name], b[name]), name
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        w = grads2[name]
        assert torch.count_nonzero(w[:, :offsets[0]]) == 0 and torch.count_nonzero(w[:, offsets[-1]:]) == 0
    # and the gradients do not read what was kept there
    c = cuda(i, cuda_device)
    kept = dict(out, errors=out["errors"].clone())
    kept["errors"][:, :offsets[0]] = float("nan")
    kept["errors"][:, offsets[-1]:] = float("nan")
    status, again = backward(c, rest["dy"].to(cuda_device), kept, o, rest["dh_final"].to(cuda_device), scale=0.3)
    assert status == 0 and all(torch.equal(again[n], grads[n]) for n in grads)
    want = delta.delta_rule_bwd(**i, dy=rest["dy"], scale=0.3, offsets=np.array(offsets), h0=rest["h0"], dh_final=rest["dh_final"])
    for name in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        close(grads2[name], want[name], name=name, terms=want.get(name + "_terms"))
