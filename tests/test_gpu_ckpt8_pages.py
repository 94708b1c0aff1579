"""GPU tests of the 8-bit activation checkpoints and the state pages.  Both
have exact results: q, scale and the 32-bit products are defined bit for bit,
and pages are moved, not computed."""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import gated

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check8(x, dev):
    q, scale = lrs.ckpt8_save(x.to(dev))
    rq, rs = gated.ckpt8(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(scale.cpu().numpy(), rs)
    v = torch.from_numpy(gated.ckpt8_values(rq, rs))
    for t in TYPES.values():
        got = lrs.ckpt8_load(q, scale, t)
        assert got.dtype == t and torch.equal(got.cpu(), v.to(t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (64,), (1, 1), (3, 63), (5, 64), (7, 65), (2, 3, 128), (129, 200),
                                   (33, 1000), (70, 1537), (2, 4, 4, 72)])
def test_ckpt8(cuda_device, shape, dtype):
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(shape[-1], generator=g))
    _check8(x.to(TYPES[dtype]), cuda_device)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ckpt8_scales_from_zero_to_the_largest(cuda_device, dtype):
    """Groups of zeros, of values too small to scale, of halves that tie, and
    of the type's largest."""
    rows = [torch.zeros(128), torch.full((128,), -0.0), torch.full((128,), 2.0 ** -101),
            torch.full((128,), 2.0 ** -100), torch.full((128,), 2.0 ** -126),
            torch.arange(128) * 0.5 + 0.0, torch.arange(-64, 64) * 1.0,
            torch.full((128,), torch.finfo(TYPES[dtype]).max),
            torch.cat([torch.full((64,), 1e30), torch.full((64,), 1e-20)])]
    rows[5][0] = 127.0     # scale 1: every odd half is a tie
    rows[5][64] = 127.0
    _check8(torch.stack(rows).to(TYPES[dtype]), cuda_device)


def test_ckpt8_of_a_group_with_nan_or_infinity(cuda_device):
    x = torch.randn(3, 130, generator=torch.Generator().manual_seed(1))
    x[0, 5], x[1, 70] = float("nan"), float("-inf")
    q, scale = lrs.ckpt8_save(x.to(cuda_device))
    v = lrs.ckpt8_load(q, scale, torch.float32).cpu()
    assert torch.isnan(v[0, :64]).all() and torch.isnan(v[1, 64:128]).all()
    clean = torch.ones(3, 130, dtype=torch.bool)
    clean[0, :64] = clean[1, 64:128] = False
    assert torch.isfinite(v[clean]).all()


def test_ckpt8_unaligned(cuda_device):
    x = torch.randn(9 * 128 + 1, generator=torch.Generator().manual_seed(2)).to(cuda_device)[1:].view(9, 128)
    q, scale = lrs.ckpt8_save(x)
    rq, rs = gated.ckpt8(x.cpu())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(scale.cpu().numpy(), rs)
    q1 = torch.empty(q.numel() + 1, dtype=torch.int8, device=cuda_device)[1:].view(q.shape).copy_(q)
    out = torch.empty(x.numel() + 1, device=cuda_device)[1:].view(x.shape)
    assert np.array_equal(lrs.ckpt8_load(q1, scale, torch.float32, out=out).cpu().numpy(),
                          gated.ckpt8_values(rq, rs))


def test_ckpt8_keeps_another_scans_activations(cuda_device):
    """The diagonal scan's gradients from its kept 8-bit activations are the
    gradients at the values they stand for."""
    import workloads
    inp = {k: v.to(cuda_device) for k, v in workloads.diag_inputs(2, 70, 64, 16, "bf16", seed=5).items()}
    dy = workloads.grad_output((2, 70, 64), 6).to(cuda_device)
    x8 = lrs.ckpt8_load(*lrs.ckpt8_save(inp["x"]))
    ref = torch.from_numpy(gated.ckpt8_values(*gated.ckpt8(inp["x"]))).to(torch.bfloat16).to(cuda_device)
    g = lrs.ssm_scan_bwd(**{**inp, "x": x8}, dy=dy)
    want = lrs.ssm_scan_bwd(**{**inp, "x": ref}, dy=dy)
    assert torch.equal(g["dx"], want["dx"]) and torch.equal(g["ddelta"], want["ddelta"])


# ---- pages ----------------------------------------------------------------------------
def _pool(layers, pages, shape, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-100, 100, (layers, pages) + shape, generator=g).to(dtype)


@pytest.mark.parametrize("layers,pages,shape,dtype", [
    (1, 1, (1,), torch.int8), (2, 9, (3,), torch.int8), (3, 40, (5, 7), torch.bfloat16),
    (1, 70, (64,), torch.float32), (2, 1100, (6,), torch.float32), (4, 2500, (1,), torch.float32),
    (2, 33, (8, 16, 32), torch.float32), (3, 20, (4099,), torch.float32)])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.8, 1.0])
def test_fork_and_compact(cuda_device, layers, pages, shape, dtype, share):
    g = torch.Generator().manual_seed(pages)
    pool = _pool(layers, pages, shape, dtype)
    used = (torch.rand(pages, generator=g) < share).to(torch.uint8)
    n = max(1, pages // 3)
    src = torch.randint(-2, pages + 2, (n,), generator=g).to(torch.int32)
    src[-1] = -1
    dev_pool, dev_used = pool.to(cuda_device), used.to(cuda_device)
    dst = lrs.state_pages_fork(dev_pool, dev_used, src.to(cuda_device), page_dim=1)
    want_used, want_dst = gated.pages_fork(used.tolist(), src.tolist())
    assert dst.cpu().tolist() == want_dst and dev_used.cpu().tolist() == want_used
    want = pool.clone()
    for s, d in zip(src.tolist(), want_dst):
        if d >= 0:
            want[:, d] = pool[:, s] if s >= 0 else 0
    assert torch.equal(dev_pool.cpu(), want)

    # some end, the rest is made dense again
    ended = torch.randint(-3, pages + 3, (pages // 2 + 1,), generator=g).to(torch.int32)
    lrs.state_pages_free(dev_used, ended.to(cuda_device))
    now = [0 if p in set(ended.tolist()) else u for p, u in enumerate(want_used)]
    assert dev_used.cpu().tolist() == now
    at = torch.randint(-2, pages + 2, (pages + 3,), generator=g).to(torch.int32)
    dev_at = at.to(cuda_device)
    moved = lrs.state_pages_compact(dev_pool, dev_used, dev_at, page_dim=1)
    want_used, want_moved, moves = gated.pages_compact(now)
    assert moved.cpu().tolist() == want_moved and dev_used.cpu().tolist() == want_used
    assert dev_at.cpu().tolist() == [p if p < 0 else want_moved[p] if p < pages else -1 for p in at.tolist()]
    after = want.clone()
    for f, t in moves:
        after[:, t] = want[:, f]
    assert torch.equal(dev_pool.cpu(), after)


def test_compact_without_a_list_and_of_a_dense_pool(cuda_device):
    pool = _pool(2, 50, (12,)).to(cuda_device)
    before = pool.clone()
    used = (torch.arange(50) < 20).to(torch.bool).to(cuda_device)
    moved = lrs.state_pages_compact(pool, used, page_dim=1)
    assert moved.cpu().tolist() == list(range(20)) + [-1] * 30
    assert torch.equal(pool, before) and used.cpu().tolist() == [True] * 20 + [False] * 30


@pytest.mark.parametrize("n", [1, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("free", [0, 700, 5000])
def test_fork_of_many_requests(cuda_device, n, free):
    """Lists longer than the planning block, more requests than free pages,
    and requests that are not valid in between."""
    pages = 6000
    g = torch.Generator().manual_seed(n + free)
    used = torch.ones(pages, dtype=torch.uint8)
    used[torch.randperm(pages, generator=g)[:free]] = 0
    src = torch.randint(-3, pages + 3, (n,), generator=g).to(torch.int32)
    pool = torch.arange(pages, dtype=torch.float32).view(pages, 1).repeat(1, 4)
    dev_pool, dev_used = pool.to(cuda_device), used.to(cuda_device)
    dst = lrs.state_pages_fork(dev_pool, dev_used, src.to(cuda_device))
    want_used, want_dst = gated.pages_fork(used.tolist(), src.tolist())
    assert dst.cpu().tolist() == want_dst and dev_used.cpu().tolist() == want_used
    for s, d in zip(src.tolist(), want_dst):
        if d >= 0:
            pool[d] = s if s >= 0 else 0
    assert torch.equal(dev_pool.cpu(), pool)


def test_pages_in_a_cuda_graph(cuda_device):
    """Free, fork and compact captured once and replayed on another pool."""
    pool, used = _pool(2, 40, (16,)).to(cuda_device), torch.zeros(40, dtype=torch.uint8, device=cuda_device)
    ended, src = (torch.zeros(3, dtype=torch.int32, device=cuda_device) for _ in range(2))
    at = torch.zeros(40, dtype=torch.int32, device=cuda_device)

    def work():
        lrs.state_pages_free(used, ended)
        dst = lrs.state_pages_fork(pool, used, src, page_dim=1)
        return dst, lrs.state_pages_compact(pool, used, at, page_dim=1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dst, moved = work()
    got = []
    for replay in (True, False):
        pool.copy_(_pool(2, 40, (16,), seed=3))
        used.copy_(torch.arange(40) % 3 == 0)
        ended.copy_(torch.tensor([3, 9, 39]))
        src.copy_(torch.tensor([0, -1, 36]))
        at.copy_(torch.arange(40))
        if replay:
            graph.replay()
        else:
            dst, moved = work()
        got.append([t.clone() for t in (pool, used, at, dst, moved)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_copy(cuda_device):
    pool = _pool(3, 30, (17,))
    src = torch.tensor([4, -1, 29, 30, 7, -2], dtype=torch.int32)
    dst = torch.tensor([5, 6, 0, 8, -1, 9], dtype=torch.int32)
    dev = pool.to(cuda_device)
    lrs.state_pages_copy(dev, src.to(cuda_device), dst.to(cuda_device), page_dim=1)
    want = pool.clone()
    want[:, 5], want[:, 6], want[:, 0] = pool[:, 4], 0, pool[:, 29]
    assert torch.equal(dev.cpu(), want)


def test_empty_lists(cuda_device):
    pool, used = _pool(1, 8, (4,)).to(cuda_device), torch.ones(8, dtype=torch.uint8, device=cuda_device)
    none = torch.empty(0, dtype=torch.int32, device=cuda_device)
    before = pool.clone()
    assert lrs.state_pages_fork(pool, used, none, page_dim=1).numel() == 0
    lrs.state_pages_copy(pool, none, none, page_dim=1)
    lrs.state_pages_free(used, none)
    used[3] = 0
    moved = lrs.state_pages_compact(pool, used, none, page_dim=1)
    assert moved.cpu().tolist() == [0, 1, 2, -1, 4, 5, 6, 3]
    before[:, 3] = before[:, 7]
    assert torch.equal(pool, before)


def test_pool_of_more_than_4_gib(cuda_device):
    """Byte offsets beyond 32 bits: pages at the two ends of a large pool."""
    pages, elems = 5000, 1 << 18
    pool = torch.empty(pages, elems, device=cuda_device)
    used = torch.zeros(pages, dtype=torch.uint8, device=cuda_device)
    used[-2:] = 1
    pool[-1], pool[-2] = 3.0, 2.0
    src = torch.tensor([pages - 1, pages - 2, -1], dtype=torch.int32, device=cuda_device)
    dst = lrs.state_pages_fork(pool, used, src)
    assert dst.cpu().tolist() == [0, 1, 2]
    assert (pool[0] == 3).all() and (pool[1] == 2).all() and (pool[2] == 0).all()
    at = src.clone()
    lrs.state_pages_free(used, dst[:1].contiguous())
    lrs.state_pages_compact(pool, used, at)
    assert at.cpu().tolist() == [3, 0, -1]
    assert (pool[0] == 2).all() and (pool[3] == 3).all()
