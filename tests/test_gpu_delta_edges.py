"""Edges of the gated delta rule on the GPU: many short sequences, offsets
beyond 32 bits, two calls at once, several host threads, bounded waits."""
import threading

import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta
from test_gpu_delta import BF, F32, check, close, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_thousand_sequences_of_a_few_tokens(cuda_device, dtype):
    lengths = torch.randint(0, 4, (1000,), generator=torch.Generator().manual_seed(1)).tolist()
    offsets = [0, *np.cumsum(lengths).tolist()]
    i, rest = inputs(1, 1, offsets[-1] + 5, 1, 2, 64, 64, dtype, n=1000)
    check(i, rest, cuda_device, offsets)


def test_step_on_a_pool_beyond_32_bits(cuda_device):
    i, _ = inputs(2, 3, 1, 4, 8, 128, 128, BF)
    i = {n: w[:, 0].contiguous() for n, w in i.items()}
    pool = torch.zeros(17000, 8, 128, 128, device=cuda_device)       # 2.2e9 elements
    pages = torch.tensor([16999, 0, 16500], dtype=torch.int32)
    before = torch.randn(3, 8, 128, 128, generator=torch.Generator().manual_seed(3))
    pool[pages.long().to(cuda_device)] = before.to(cuda_device)
    y = lrs.delta_rule_step(**cuda(i, cuda_device), states=pool, pages=pages.to(cuda_device))
    want, after = delta.delta_rule_step(**i, states=before, pages=None)
    close(y, want)
    close(pool[pages.long().to(cuda_device)], after)
    assert torch.count_nonzero(pool[1:16500]) == 0


def test_tokens_beyond_32_bits(cuda_device):
    """More than 2^31 elements in v and y; decays so fast that the end does not see the beginning."""
    L, H, tail = 540000, 32, 640
    g = torch.Generator(device=cuda_device).manual_seed(4)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=cuda_device, dtype=BF)

    q, k = rand(1, L, 1, 128) / 11.3, rand(1, L, 1, 128) / 11.3
    v, gate = rand(1, L, H, 128), -torch.rand(1, L, H, generator=g, device=cuda_device).to(BF) - 0.5
    beta = torch.rand(1, L, H, generator=g, device=cuda_device).to(BF)
    assert v.numel() > 2 ** 31
    y, hf = lrs.delta_rule_fwd(q, k, v, gate, beta, return_final_state=True)
    last = [w[:, -tail:].contiguous() for w in (q, k, v, gate, beta)]
    y2, hf2 = lrs.delta_rule_fwd(*last, return_final_state=True)
    # e^(-0.5 * 384) and less of what came before is left
    close(y[:, -256:], y2[:, -256:].double().cpu().numpy(), BF)
    close(hf, hf2.double().cpu().numpy(), F32)
    lrs.ssm_check_device_errors()


def test_two_calls_at_once(cuda_device):
    sets = []
    for seed in (5, 6):
        i, rest = inputs(seed, 2, 700, 2, 4, 128, 64, BF)
        sets.append((cuda(i, cuda_device), rest["dy"].to(cuda_device)))

    def both(c, dy):
        y, saved = lrs.delta_rule_fwd(**c, save="states")
        w = {n: t for n, t in c.items() if n != "v"}
        return [y, *lrs.delta_rule_bwd(**w, dy=dy, saved=saved).values()]

    alone = [both(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(both(*s))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    # and from two host threads, sizes of different shared memory
    i, _ = inputs(7, 1, 200, 1, 2, 16, 16, F32)
    small = cuda(i, cuda_device)
    want = lrs.delta_rule_fwd(**small)
    bad = []

    def call(which):
        try:
            with torch.cuda.stream(streams[which]):
                for _ in range(20):
                    if which:
                        ok = all(torch.equal(x, y) for x, y in zip(alone[0], both(*sets[0])))
                    else:
                        ok = torch.equal(want, lrs.delta_rule_fwd(**small))
                    if not ok:
                        bad.append(which)
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=call, args=(w,)) for w in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


def test_a_wait_that_runs_out_is_reported(cuda_device):
    stream = torch.cuda.current_stream().cuda_stream
    lrs.ssm_check_device_errors()
    assert lrs.library().delta_selftest_wait_timeout(stream) == 0
    with pytest.raises(lrs.SsmError):
        lrs.ssm_check_device_errors()
    lrs.ssm_check_device_errors()
    i, rest = inputs(8, 1, 100, 1, 1, 64, 64, BF)
    check(i, rest, cuda_device)


def test_page_calls_on_the_rule_s_pool(cuda_device):
    """Fork and compact pages of matrix states between tokens."""
    i, _ = inputs(9, 4, 3, 1, 2, 64, 64, BF)
    pool = torch.zeros(8, 2, 64, 64, device=cuda_device)
    used = torch.zeros(8, dtype=torch.uint8, device=cuda_device)
    new = lrs.state_pages_fork(pool, used, torch.full((2,), -1, dtype=torch.int32, device=cuda_device))
    token = lambda t, rows: {n: w[rows, t].contiguous().to(cuda_device) for n, w in i.items()}  # noqa: E731
    lrs.delta_rule_step(**token(0, slice(0, 2)), states=pool, pages=new)
    twice = torch.cat((new, lrs.state_pages_fork(pool, used, new)))
    y = lrs.delta_rule_step(**token(1, slice(0, 4)), states=pool, pages=twice)
    # row 2 continues row 0's first token
    one = {n: torch.stack((w[0, 0], w[2, 1]))[None] for n, w in i.items()}
    close(y[2:3], delta.delta_rule(**one)["y"][:, 1])
    lrs.state_pages_free(used, new)
    pages = twice[2:].clone()
    lrs.state_pages_compact(pool, used, pages)
    assert sorted(pages.tolist()) == [0, 1]
    y = lrs.delta_rule_step(**token(2, slice(2, 4)), states=pool, pages=pages)
    three = {n: torch.stack((w[0, 0], w[2, 1], w[2, 2]))[None] for n, w in i.items()}
    close(y[:1], delta.delta_rule(**three)["y"][:, 2])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (40, 24), (20, 33)])
@pytest.mark.parametrize("L,at", [(100, 10), (200, 64), (200, 75), (130, 129), (2000, 5), (2000, 1100)])
def test_a_step_without_decay_left_drops_a_nan_state_wherever_it_lies(cuda_device, dtype, K, V, L, at):
    i, rest = inputs(10, 2, L, 1, 2, K, V, dtype)
    i["g"][:, at, 0] = float("-inf")
    h0 = torch.full_like(rest["h0"], float("nan"))
    y, hf = lrs.delta_rule_fwd(**cuda(i, cuda_device), h0=h0.to(cuda_device), return_final_state=True)
    want = delta.delta_rule(**{n: w[:, at:].contiguous() for n, w in i.items()})
    close(y[:, at:, :1], want["y"][:, :, :1], terms=want["y_terms"][:, :, :1])
    close(hf[:, 0], want["h_final"][:, 0])
    # before it, and in the head without such a step, the NaN stands
    assert torch.isnan(y[:, :at]).all() and torch.isnan(y[:, :, 1]).all() and torch.isnan(hf[:, 1]).all()


def test_many_sequences_of_one_part(cuda_device):
    """So many steps that sequences are taken in parts, and none longer than a part."""
    i, rest = inputs(11, 1, 2048, 1, 2, 64, 64, BF, n=8)
    check(i, rest, cuda_device, [256 * n for n in range(9)], h0=False)
    check(i, rest, cuda_device, [0, 0, 0, 0, 1, 1, 1, 500, 501])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("g", [-101.0, float("-inf")])
def test_a_token_without_decay_left_drops_a_nan_state(cuda_device, dtype, g):
    i, _ = inputs(12, 2, 1, 1, 2, 64, 64, dtype)
    i = {n: w[:, 0].contiguous() for n, w in i.items()}
    i["g"].fill_(g)
    pool = torch.full((2, 2, 64, 64), float("nan"), device=cuda_device)
    y = lrs.delta_rule_step(**cuda(i, cuda_device), states=pool)
    want, after = delta.delta_rule_step(**i, states=torch.zeros(2, 2, 64, 64), pages=None)
    close(y, want)
    close(pool, after)


def test_parts_on_another_stream_and_in_a_graph(cuda_device):
    """A long sequence of few heads: four kernels that begin while the one before runs."""
    i, rest = inputs(13, 1, 2500, 1, 2, 128, 64, BF, n=3)
    c, h0 = cuda(i, cuda_device), rest["h0"].to(cuda_device)
    o = torch.tensor([0, 700, 700, 2490], dtype=torch.int32, device=cuda_device)
    call = lambda: lrs.delta_rule_fwd(**c, offsets=o, h0=h0, return_final_state=True)  # noqa: E731
    first = call()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = [call() for _ in range(3)]
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = call()
    for _ in range(3):
        for t in third:
            t.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for out in (*second, third):
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("offsets", [[0, 2400, 100, 2000, 10 ** 9], [-5, 2500, 0, 2500, 0], [2000, 1500, 1000, 500, 0]])
def test_bad_offsets_of_long_sequences_touch_nothing_outside(cuda_device, offsets):
    i, rest = inputs(14, 1, 2500, 1, 2, 64, 64, BF, n=4)
    o = torch.tensor(offsets, dtype=torch.int32, device=cuda_device)
    c = cuda(i, cuda_device)
    room = torch.full((4096 + 2500 * 2 * 64 + 4096,), 7.0, dtype=BF, device=cuda_device)
    lrs.delta_rule_fwd(**c, offsets=o, h0=rest["h0"].to(cuda_device), return_final_state=True,
                       y=room[4096:-4096].view(1, 2500, 2, 64))
    torch.cuda.synchronize()
    assert torch.all(room[:4096] == 7.0) and torch.all(room[-4096:] == 7.0)
    lrs.ssm_check_device_errors()
