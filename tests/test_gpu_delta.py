"""The gated delta rule on the GPU against the fp64 oracle.

Bounds, from the formats alone.  fp32: sums of at most a few hundred terms and
64 steps a block, 2^-24 each: 1e-5 in the 2-norm.  bf16: up to five independent
roundings of at most 2^-8 (operands and the output itself), uniform in size:
sqrt(5) 2^-8 / sqrt(3) = 5.05e-3 in the 2-norm; single elements stay within
40 2^-8 / 8 = 2e-2 of the largest.  fp32 results of bf16 inputs (states and
their gradients) rest on operands of 16 bits: sqrt(5) 2^-17 / sqrt(3) = 1e-5.

These bounds are relative to the result where it is no smaller than its terms.
A sum of rounded terms, sum_i a_i with errors delta a_i independent of one
another, is off by delta (sum_i a_i^2)^(1/2), whatever is left of the sum: the
oracle gives that 2-norm of the terms beside the sums (over the states' rows,
and over the writes of a block, which pile up where keys are alike), and the
bound is delta times the value and the terms.
"""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta

pytestmark = pytest.mark.gpu

TWO_NORM = {torch.float32: 1e-5, torch.bfloat16: 5.05e-3}
LARGEST = {torch.float32: 1e-4, torch.bfloat16: 2e-2}
BF, F32 = torch.bfloat16, torch.float32


def inputs(seed, Bs, L, G, H, K, V, dtype, n=None, decay=0.05):
    g = torch.Generator().manual_seed(seed)
    n = Bs if n is None else n

    def unit(*shape):
        w = torch.randn(*shape, generator=g) + 0.3
        return (w / w.norm(dim=-1, keepdim=True)).to(dtype)

    i = dict(q=unit(Bs, L, G, K), k=unit(Bs, L, G, K), v=torch.randn(Bs, L, H, V, generator=g).to(dtype),
             g=(-decay * torch.rand(Bs, L, H, generator=g)).to(dtype),
             beta=torch.rand(Bs, L, H, generator=g).to(dtype))
    rest = dict(h0=0.3 * torch.randn(n, H, V, K, generator=g), dy=torch.randn(Bs, L, H, V, generator=g).to(dtype),
                dh_final=torch.randn(n, H, V, K, generator=g))
    return i, rest


def close(got, want, dtype=None, name="", terms=None):
    """``terms``: the size of the terms that each value is the sum of."""
    dtype = got.dtype if dtype is None else dtype
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)), name
    size = np.linalg.norm(want) + (0.0 if terms is None else np.linalg.norm(terms))
    assert np.linalg.norm(got - want) <= TWO_NORM[dtype] * size + 1e-30, (name, np.linalg.norm(got - want) / size)
    if want.size:
        top = np.max(np.abs(want)) + (0.0 if terms is None else np.max(terms))
        assert np.max(np.abs(got - want)) <= LARGEST[dtype] * top + 1e-30, name


def cuda(d, dev):
    return {k: None if v is None else v.to(dev) for k, v in d.items()}


def check(i, rest, dev, offsets=None, h0=True, dend=True, scale=None):
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=dev)
    h = rest["h0"] if h0 else None
    d = rest["dh_final"] if dend else None
    c = cuda(i, dev)
    y, hf, saved = lrs.delta_rule_fwd(**c, scale=scale, offsets=o, h0=None if h is None else h.to(dev),
                                      return_final_state=True, save="states")
    want = delta.delta_rule(**i, scale=scale, offsets=offsets if offsets is None else np.array(offsets), h0=h)
    close(y, want["y"], name="y", terms=want["y_terms"])
    close(hf, want["h_final"], name="h_final")
    v = c.pop("v")
    got = lrs.delta_rule_bwd(**c, dy=rest["dy"].to(dev), saved=saved, scale=scale, offsets=o,
                             dh_final=None if d is None else d.to(dev))
    assert v is not None
    want = delta.delta_rule_bwd(**i, dy=rest["dy"], scale=scale,
                                offsets=offsets if offsets is None else np.array(offsets), h0=h, dh_final=d)
    for name in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        close(got[name], want[name], name=name, terms=want.get(name + "_terms"))
    lrs.ssm_check_device_errors()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Bs,L,G,H,K,V", [
    (1, 1, 1, 1, 64, 64), (2, 63, 1, 2, 128, 64), (1, 64, 2, 2, 128, 128), (2, 65, 2, 4, 64, 64),
    (1, 130, 1, 1, 16, 16), (1, 200, 1, 3, 96, 40), (3, 77, 2, 2, 1, 1), (1, 70, 1, 1, 5, 3), (1, 100, 1, 2, 20, 33),
    (1, 129, 1, 1, 256, 256), (1, 66, 1, 1, 200, 8), (2, 300, 2, 6, 128, 64), (1, 90, 1, 1, 24, 72), (1, 68, 1, 2, 72, 136),
])
def test_sizes(cuda_device, dtype, Bs, L, G, H, K, V):
    i, rest = inputs(L + K + V, Bs, L, G, H, K, V, dtype)
    check(i, rest, cuda_device)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(128, 64), (64, 64), (40, 24)])
@pytest.mark.parametrize("offsets", [[0, 5, 5, 133, 262], [3, 67, 68, 200, 200], [0, 0, 262], [0, 64, 128, 262],
                                     [0, 1, 2, 3, 4, 5, 261]])
def test_packed(cuda_device, dtype, K, V, offsets):
    i, rest = inputs(7, 1, 262, 2, 4, K, V, dtype, n=len(offsets) - 1)
    check(i, rest, cuda_device, offsets)


@pytest.mark.parametrize("K,V", [(128, 64), (64, 128), (40, 24)])
@pytest.mark.parametrize("Bs,L,offsets,h0", [(1, 2100, None, True), (2, 1537, None, False), (1, 3000, [0, 0, 2000, 2001, 2900], True),
                                             (1, 2500, [100, 612, 612, 2500], False)])
def test_long_sequences_of_few_heads(cuda_device, K, V, Bs, L, offsets, h0):
    """Taken in parts that are joined afterwards."""
    i, rest = inputs(16, Bs, L, 1, 2, K, V, BF, n=None if offsets is None else len(offsets) - 1, decay=0.02)
    check(i, rest, cuda_device, offsets, h0=h0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("h0,dend", [(False, False), (True, False), (False, True)])
def test_optional_states(cuda_device, dtype, h0, dend):
    i, rest = inputs(3, 2, 150, 1, 2, 128, 64, dtype)
    check(i, rest, cuda_device, h0=h0, dend=dend, scale=0.7)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("decay", [0.0, 1.0, 30.0, 300.0])
def test_decays(cuda_device, dtype, decay):
    """None at all, ordinary, so fast that a few steps forget, and below what fp32 holds."""
    i, rest = inputs(4, 1, 140, 1, 2, 64, 64, dtype, decay=decay)
    check(i, rest, cuda_device)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_alike_keys_and_full_writes(cuda_device, dtype):
    """The block's system at its worst: every key the same, beta = 1."""
    i, rest = inputs(5, 1, 128, 1, 2, 64, 64, dtype)
    i["k"] = i["k"][:, :1].expand_as(i["k"]).contiguous()
    i["beta"] = torch.ones_like(i["beta"])
    o = lrs.delta_rule_fwd(**cuda(i, cuda_device), return_final_state=True)
    want = delta.delta_rule(**i)
    close(o[0], want["y"], terms=want["y_terms"])
    # the state is a sum of cancelling writes; measured against the values written
    err = np.linalg.norm(o[1].double().cpu().numpy() - want["h_final"])
    assert err <= 1e-5 * np.linalg.norm(i["v"].double().numpy())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_step_without_decay_left_drops_a_nan_state(cuda_device, dtype):
    i, rest = inputs(6, 2, 100, 1, 2, 64, 64, dtype)
    i["g"][:, 0] = float("-inf")
    h0 = torch.full_like(rest["h0"], float("nan")).to(cuda_device)
    y, hf = lrs.delta_rule_fwd(**cuda(i, cuda_device), h0=h0, return_final_state=True)
    want = delta.delta_rule(**i)
    close(y, want["y"], terms=want["y_terms"])
    close(hf, want["h_final"])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_nan_stays_in_its_sequence_and_head(cuda_device, dtype):
    i, rest = inputs(8, 1, 200, 2, 2, 64, 64, dtype, n=3)
    offsets = torch.tensor([0, 70, 130, 200], dtype=torch.int32, device=cuda_device)
    c = cuda(i, cuda_device)
    whole = lrs.delta_rule_fwd(**c, offsets=offsets)
    c["v"][0, 75, 1] = float("nan")
    c["k"][0, 90, 1] = float("inf")
    y = lrs.delta_rule_fwd(**c, offsets=offsets)
    assert torch.equal(y[:, :70], whole[:, :70]) and torch.equal(y[:, 130:], whole[:, 130:])
    assert torch.equal(y[:, :, 0], whole[:, :, 0])
    assert torch.isnan(y[0, 130 - 1, 1]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(128, 64), (64, 128), (36, 20)])
def test_parts_of_a_sequence(cuda_device, dtype, K, V):
    """A sequence in two calls, the second from the first's state, and token by token from a page."""
    i, _ = inputs(9, 2, 141, 1, 2, K, V, dtype)
    c = cuda(i, cuda_device)
    y, hf = lrs.delta_rule_fwd(**c, return_final_state=True)
    part = lambda a, b: {n: w[:, a:b].contiguous() for n, w in c.items()}  # noqa: E731
    y1, h1 = lrs.delta_rule_fwd(**part(0, 77), return_final_state=True)
    y2, h2 = lrs.delta_rule_fwd(**part(77, 141), h0=h1, return_final_state=True)
    close(torch.cat((y1, y2), 1), y.double().cpu().numpy(), dtype)
    close(h2, hf.double().cpu().numpy(), F32)
    states = torch.zeros(5, *h1.shape[1:], device=cuda_device)
    pages = torch.tensor([3, 1], dtype=torch.int32, device=cuda_device)
    states[pages.long()] = h1
    for t in range(77, 141):
        y3 = lrs.delta_rule_step(**{n: w[:, t].contiguous() for n, w in c.items()}, states=states, pages=pages)
        close(y3, y[:, t].double().cpu().numpy(), dtype)
    close(states[pages.long()], hf.double().cpu().numpy(), F32)
    assert torch.count_nonzero(states[[0, 2, 4]]) == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Bs,G,H,K,V", [(1, 1, 1, 128, 64), (7, 2, 4, 64, 64), (3, 1, 2, 128, 128), (2, 1, 1, 96, 40),
                                        (2, 1, 3, 5, 3), (1, 1, 1, 256, 256), (2, 2, 2, 255, 9), (4, 1, 1, 16, 100)])
def test_step(cuda_device, dtype, Bs, G, H, K, V):
    i, rest = inputs(10, Bs, 1, G, H, K, V, dtype)
    i = {n: w[:, 0].contiguous() for n, w in i.items()}
    states = torch.randn(Bs + 3, H, V, K, generator=torch.Generator().manual_seed(1))
    pages = torch.randperm(Bs + 3, generator=torch.Generator().manual_seed(2))[:Bs].to(torch.int32)
    if Bs > 2:
        pages[1], pages[2] = -1, Bs + 3
    pool = states.to(cuda_device)
    y = lrs.delta_rule_step(**cuda(i, cuda_device), states=pool, pages=pages.to(cuda_device))
    want, after = delta.delta_rule_step(**i, states=states, pages=pages)
    close(y, want)
    close(pool, after)
    idle = [p for p in range(Bs + 3) if p not in pages.tolist()]
    assert torch.equal(pool[idle].cpu(), states[idle])
    # row b uses page b
    pool = states.to(cuda_device)
    y = lrs.delta_rule_step(**cuda(i, cuda_device), states=pool)
    want, after = delta.delta_rule_step(**i, states=states, pages=None)
    close(y, want)
    close(pool, after)


def test_step_on_states_off_16_bytes(cuda_device):
    i, _ = inputs(11, 2, 1, 1, 2, 64, 64, BF)
    i = {n: w[:, 0].contiguous() for n, w in i.items()}
    room = torch.randn(2 * 2 * 64 * 64 + 1, generator=torch.Generator().manual_seed(1))
    pool = room.to(cuda_device)[1:].view(2, 2, 64, 64)
    before = pool.cpu().clone()
    y = lrs.delta_rule_step(**cuda(i, cuda_device), states=pool)
    want, after = delta.delta_rule_step(**i, states=before, pages=None)
    close(y, want)
    close(pool, after)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_inputs_off_16_bytes(cuda_device, dtype):
    i, rest = inputs(12, 1, 130, 1, 2, 64, 64, dtype)
    c = {}
    for n, w in i.items():
        room = torch.zeros(w.numel() + 1, dtype=dtype, device=cuda_device)
        room[1:] = w.flatten().to(cuda_device)
        c[n] = room[1:].view(w.shape)
    got, saved = lrs.delta_rule_fwd(**c, save="states")
    want = delta.delta_rule(**i)
    close(got, want["y"], terms=want["y_terms"])
    c.pop("v")
    grads = lrs.delta_rule_bwd(**c, dy=rest["dy"].to(cuda_device), saved=saved)
    want = delta.delta_rule_bwd(**i, dy=rest["dy"])
    for name in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        close(grads[name], want[name], name=name, terms=want.get(name + "_terms"))


@pytest.mark.parametrize("offsets", [[5, 3, 300, 2, 90], [-7, 40, 10 ** 9, 10 ** 9, 2 ** 31 - 1], [90, 60, 30, 10, 0],
                                     [-1, -1, -1, -1, -1]])
def test_bad_offsets_touch_nothing_outside(cuda_device, offsets):
    """Whatever the offsets hold, rows before and behind the tensors stay."""
    i, rest = inputs(13, 1, 90, 1, 2, 64, 64, BF, n=4)
    o = torch.tensor(offsets, dtype=torch.int32, device=cuda_device)
    c = cuda(i, cuda_device)
    room = torch.full((4096 + 90 * 2 * 64 + 4096,), 7.0, dtype=BF, device=cuda_device)
    y = room[4096:-4096].view(1, 90, 2, 64)
    _, saved = lrs.delta_rule_fwd(**c, offsets=o, save="states", y=y)
    c.pop("v")
    lrs.delta_rule_bwd(**c, dy=rest["dy"].to(cuda_device), saved=saved, offsets=o)
    torch.cuda.synchronize()
    assert torch.all(room[:4096] == 7.0) and torch.all(room[-4096:] == 7.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(128, 64), (64, 64)])
def test_same_bits_on_another_stream_and_in_a_graph(cuda_device, dtype, K, V):
    i, rest = inputs(14, 2, 333, 2, 4, K, V, dtype)
    c, dy = cuda(i, cuda_device), rest["dy"].to(cuda_device)
    h0 = rest["h0"].to(cuda_device)

    def both():
        y, hf, saved = lrs.delta_rule_fwd(**c, h0=h0, return_final_state=True, save="states")
        w = {n: t for n, t in c.items() if n != "v"}
        return (y, hf, *lrs.delta_rule_bwd(**w, dy=dy, saved=saved, dh_final=hf).values())

    first = [t.clone() for t in both()]
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = both()
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    for _ in range(2):
        for t in third:
            t.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_refusals_of_the_binding(cuda_device):
    i, rest = inputs(15, 1, 20, 2, 4, 16, 8, BF)
    c = cuda(i, cuda_device)
    o = torch.tensor([0, 20], dtype=torch.int32, device=cuda_device)
    for bad in (dict(q=c["q"].float()), dict(k=c["k"][:, :10]), dict(v=c["v"].transpose(1, 2)), dict(g=c["g"][..., :3]),
                dict(beta=c["beta"].cpu()), dict(q=c["q"][..., :1, :].expand(1, 20, 3, 16)), dict(offsets=o.long()),
                dict(offsets=o[:1]), dict(h0=torch.zeros(1, 4, 16, 8, device=cuda_device)), dict(save="8bit"),
                dict(y=torch.zeros(1, 20, 4, 8, device=cuda_device)), dict(v=None), dict(scale=float("nan"))):
        with pytest.raises((TypeError, ValueError, lrs.SsmError)):
            lrs.delta_rule_fwd(**{**c, **bad})
    two = {n: torch.cat((w, w)) for n, w in c.items()}
    with pytest.raises(ValueError):
        lrs.delta_rule_fwd(**two, offsets=o)
    y, saved = lrs.delta_rule_fwd(**c, save="states")
    w = {n: t for n, t in c.items() if n != "v"}
    for bad in (dict(saved={}), dict(saved=dict(saved, states=None)), dict(saved=dict(saved, errors=y.float())),
                dict(dy=y[..., :4]), dict(dh_final=y)):
        with pytest.raises((TypeError, ValueError, lrs.SsmError)):
            lrs.delta_rule_bwd(**{**w, "dy": y, "saved": saved, **bad})
    t = {n: x[:, 0].contiguous() for n, x in c.items()}
    for bad in (dict(states=torch.zeros(2, 4, 16, 8, device=cuda_device)), dict(states=None),
                dict(states=torch.zeros(2, 4, 8, 16, device=cuda_device, dtype=BF)),
                dict(pages=torch.zeros(2, dtype=torch.int32, device=cuda_device)),
                dict(states=torch.zeros(0, 4, 8, 16, device=cuda_device))):
        with pytest.raises((TypeError, ValueError, lrs.SsmError)):
            lrs.delta_rule_step(**{**t, "states": torch.zeros(2, 4, 8, 16, device=cuda_device), **bad})
