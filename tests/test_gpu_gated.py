"""GPU parity of the gated linear recurrence against the fp64 oracle.

Error bounds.  A step's decay has a relative error of at most ~8 * 2^-24
(exponential, its argument's rounding, the gate), so after n steps a state
is off by at most n * 2^-21 of the largest state, and a step's input by a few
2^-22 of its own; 16 covers the latter.  tol(n) = (16 + n) * 2^-21 of the
scale, n capped at the sequence length.  A gradient joins two such scans:
twice that, of the size of its terms.  bf16 outputs add one rounding, 2^-8 of
the value (half an ulp is 2^-9; the factor 2 covers a neighbour that rounds
the other way).
"""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import gated

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = [(1, 1, 1), (1, 1, 64), (3, 2, 7), (2, 63, 64), (2, 64, 65), (2, 65, 70), (1, 129, 200),
         (3, 200, 33), (2, 513, 128), (1, 1030, 72), (5, 96, 1536), (1, 4200, 64)]


def case(Bs, L, ED, dtype, seed, resets=False, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    inp = {k: torch.randn(Bs, L, ED, generator=g).to(t) for k in ("x", "gate_r", "gate_i")}
    a = 0.9 + 0.099 * torch.rand(ED, generator=g)
    inp["lam"] = torch.log(torch.expm1(-torch.log(a) / 8.0))
    reset = (torch.rand(Bs, L, generator=g) < 0.03).to(torch.uint8) if resets else None
    more = dict(h0=torch.randn(Bs, ED, generator=g), dy=torch.randn(Bs, L, ED, generator=g).to(t),
                dh_final=torch.randn(Bs, ED, generator=g))
    return inp, reset, more


def on(d, dev):
    return {k: (v.to(dev) if v is not None else None) for k, v in d.items()}


def near(got, ref, tol, dtype, what):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, what
    bound = tol + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3e (bound %.3e)" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(g - ref)), np.max(bound))


def tol_state(L, ref):
    return (16 + L) * 2.0 ** -21 * max(1.0, float(np.max(np.abs(ref))))


def check_fwd(inp, reset, h0, dtype, dev, save="states"):
    L = inp["x"].shape[1]
    ref = gated.gated_scan(**inp, reset=reset, h0=h0)
    r = None if reset is None else reset.to(dev)
    y, hf, saved = lrs.gated_scan_fwd(**on(inp, dev), reset=r, h0=None if h0 is None else h0.to(dev),
                                      return_final_state=True, save=save)
    tol = tol_state(L, ref)
    assert y.dtype == inp["x"].dtype and hf.dtype == torch.float32
    near(y, ref, tol, dtype, "y")
    near(hf, ref[:, -1], tol, "f32", "h_final")
    near(saved["states"], gated.kept_states(ref, h0), tol, "f32", "states")
    return y, hf, saved


def check_bwd(inp, reset, more, dtype, dev, saved, values=None):
    """`values`: what the 8-bit checkpoints stand for."""
    L = inp["x"].shape[1]
    dh = more["dh_final"]
    g = lrs.gated_scan_bwd(*([None] * 3 if values else [inp[k].to(dev) for k in ("x", "gate_r", "gate_i")]),
                           inp["lam"].to(dev), more["dy"].to(dev), saved,
                           reset=None if reset is None else reset.to(dev),
                           dh_final=None if dh is None else dh.to(dev))
    src = values or inp
    ref = gated.gated_scan_bwd(src["x"], src["gate_r"], src["gate_i"], inp["lam"], more["dy"],
                               saved["states"], reset=reset, dh_final=dh)
    rel = 2 * (16 + L) * 2.0 ** -21
    gmax = max(1.0, float(np.max(np.abs(ref["dh0"]))), float(np.max(np.abs(ref["dx"]))))
    xmax = max(1.0, float(np.max(np.abs(gated.f64(src["x"])))))
    near(g["dx"], ref["dx"], rel * gmax, dtype, "dx")
    near(g["dgate_i"], ref["dgate_i"], rel * gmax * xmax, dtype, "dgate_i")
    near(g["dgate_r"], ref["dgate_r"], rel * max(1.0, float(ref["size"].max())), dtype, "dgate_r")
    near(g["dlam"], ref["dlam"], rel * max(1.0, float(ref["size_lam"].max())), "f32", "dlam")
    near(g["dh0"], ref["dh0"], rel * gmax, "f32", "dh0")
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,L,ED", SIZES)
@pytest.mark.parametrize("resets", [False, True])
def test_forward_and_backward(cuda_device, Bs, L, ED, dtype, resets):
    inp, reset, more = case(Bs, L, ED, dtype, seed=L + ED, resets=resets)
    _, _, saved = check_fwd(inp, reset, more["h0"] if resets else None, dtype, cuda_device)
    check_bwd(inp, reset, more if resets else dict(more, dh_final=None), dtype, cuda_device, saved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,L,ED", [(1, 1, 1), (2, 64, 64), (2, 65, 70), (1, 129, 200), (3, 200, 33),
                                     (2, 513, 128), (1, 700, 1536)])
def test_8bit_checkpoints(cuda_device, Bs, L, ED, dtype):
    """What the forward keeps is ckpt8_save's, bit for bit; the backward's
    gradients are those at the values it stands for."""
    inp, reset, more = case(Bs, L, ED, dtype, seed=7 * L + ED, resets=True)
    y, hf, saved = check_fwd(inp, reset, None, dtype, cuda_device, save="8bit")
    y2, hf2 = lrs.gated_scan_fwd(**on(inp, cuda_device), reset=reset.to(cuda_device), return_final_state=True)
    assert torch.equal(y, y2) and torch.equal(hf, hf2)
    values = {}
    for k, q in (("x", "x"), ("gate_r", "r"), ("gate_i", "i")):
        rq, rs = gated.ckpt8(inp[k])
        assert np.array_equal(saved[q + "_q"].cpu().numpy(), rq)
        assert np.array_equal(saved[q + "_s"].cpu().numpy(), rs)
        values[k] = gated.ckpt8_values(rq, rs)
    check_bwd(inp, reset, more, dtype, cuda_device, saved, values)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ED", [128, 136, 131])
def test_8bit_checkpoints_of_special_values(cuda_device, ED, dtype):
    """NaN, infinities, zeros and tiny values: the forward still keeps what
    ckpt8_save does, bit for bit."""
    inp, _, _ = case(2, 70, ED, dtype, seed=ED)
    for k, at in (("x", 0), ("gate_r", 1), ("gate_i", 2)):
        v = inp[k]
        v[0, at, 5] = float("nan")
        v[0, 3 + at, 64] = float("inf")
        v[1, 6 + at, 63] = -float("inf")
        v[1, 9 + at] = -0.0
        v[1, 12 + at] = v[1, 12 + at] * 2.0 ** -105
        v[1, 15 + at, 7] = 3e38
        v[0, 69, 1 + at] = -float("nan")
    d = on(inp, cuda_device)
    _, saved = lrs.gated_scan_fwd(**d, save="8bit")
    for k, q in (("x", "x"), ("gate_r", "r"), ("gate_i", "i")):
        rq, rs = lrs.ckpt8_save(d[k])
        assert torch.equal(saved[q + "_s"].view(torch.int32).flatten(), rs.view(torch.int32).flatten())
        assert torch.equal(saved[q + "_q"].flatten(), rq.flatten())


def test_gradients_against_differences(cuda_device):
    """Directional differences of the forward kernel itself, in fp32.  With a
    step of 2^-6 the truncation is O(2^-12) of the loss' third derivative and
    the rounding 2^-21 * 64 of its size: 2 % of the derivative's scale."""
    Bs, L, ED = 2, 150, 96
    inp, reset, more = case(Bs, L, ED, "f32", seed=5, resets=True)
    d = on(inp, cuda_device)
    r, h0 = reset.to(cuda_device), more["h0"].to(cuda_device)
    w, wf = more["dy"].to(cuda_device), more["dh_final"].to(cuda_device)

    def loss(**kw):
        y, hf = lrs.gated_scan_fwd(**{**d, **{k: v for k, v in kw.items() if k != "h0"}}, reset=r,
                                   h0=kw.get("h0", h0), return_final_state=True)
        return ((y.double() * w).sum() + (hf.double() * wf).sum()).item()

    _, saved = lrs.gated_scan_fwd(**d, reset=r, h0=h0, save="states")
    g = lrs.gated_scan_bwd(d["x"], d["gate_r"], d["gate_i"], d["lam"], w, saved, reset=r, dh_final=wf)
    eps = 2.0 ** -6
    gen = torch.Generator().manual_seed(9)
    for name, grad in (("x", "dx"), ("gate_r", "dgate_r"), ("gate_i", "dgate_i"), ("lam", "dlam"), ("h0", "dh0")):
        base = h0 if name == "h0" else d[name]
        v = torch.randn(base.shape, generator=gen).to(cuda_device)
        num = (loss(**{name: base + eps * v}) - loss(**{name: base - eps * v})) / (2 * eps)
        ana = (g[grad].double() * v.double()).sum().item()
        scale = (g[grad].double().norm() * v.double().norm() / v.numel() ** 0.5).item()
        assert abs(num - ana) <= 0.02 * max(scale, abs(ana)), (name, num, ana, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_reset_drops_infinities_and_nan(cuda_device, dtype):
    Bs, L, ED = 2, 300, 130
    inp, _, more = case(Bs, L, ED, dtype, seed=1)
    reset = torch.zeros(Bs, L, dtype=torch.bool)
    reset[0, 100] = reset[1, 1] = reset[1, 299] = True
    bad = {k: v.clone() for k, v in inp.items()}
    bad["x"][0, 99] = float("nan")
    bad["x"][0, 3, 5] = float("inf")
    h0 = torch.full((Bs, ED), float("inf"))
    d = on(bad, cuda_device)
    y, hf, saved = lrs.gated_scan_fwd(**d, reset=reset.to(cuda_device), h0=h0.to(cuda_device),
                                      return_final_state=True, save="states")
    good = {k: v.clone() for k, v in inp.items()}
    ref = gated.gated_scan(**good, reset=reset, h0=torch.zeros(Bs, ED))
    tol = tol_state(L, ref)
    near(y[0, 100:], ref[0, 100:], tol, dtype, "after the first reset")
    near(y[1, 1:], ref[1, 1:], tol, dtype, "after the second row's reset")
    near(hf, ref[:, -1], tol, "f32", "h_final")
    # gradients: dy that is NaN in the next document stays there
    dy = more["dy"].clone()
    dy[0, 100:] = float("nan")
    fine = on(good, cuda_device)
    _, saved = lrs.gated_scan_fwd(**fine, reset=reset.to(cuda_device), save="states")
    g = lrs.gated_scan_bwd(fine["x"], fine["gate_r"], fine["gate_i"], fine["lam"], dy.to(cuda_device), saved,
                           reset=reset.to(cuda_device), dh_final=h0.to(cuda_device))
    for k in ("dx", "dgate_r", "dgate_i"):
        assert torch.isfinite(g[k][0, :100]).all(), k
        assert torch.isfinite(g[k][1, :299]).all(), k
    assert torch.isfinite(g["dh0"]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates(cuda_device, dtype):
    """Gates that are fully open or shut, and decays of 0 and 1: all outputs
    and gradients are finite and follow the formula (m -> 0 with la)."""
    L = 70
    r = torch.tensor([-200.0, -90.0, -30.0, 0.0, 30.0, 200.0, float("-inf"), float("inf")])
    inp = dict(x=torch.randn(1, L, 64, generator=torch.Generator().manual_seed(2)),
               gate_r=r.repeat(8).expand(1, L, 64).clone(),
               gate_i=r.repeat_interleave(8).expand(1, L, 64).clone(),
               lam=torch.tensor([-150.0, -50.0, -3.0, 0.0, 3.0, 25.0, 60.0, 1.0]).repeat(8).roll(3))
    inp = {k: (v.to(TYPES[dtype]).contiguous() if k != "lam" else v) for k, v in inp.items()}
    _, _, more = case(1, L, 64, dtype, seed=4)
    _, _, saved = check_fwd(inp, None, more["h0"], dtype, cuda_device)
    check_bwd(inp, None, more, dtype, cuda_device, saved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_of_a_sequence(cuda_device, dtype):
    """A sequence scanned in parts, each from the last one's final state."""
    inp, reset, more = case(2, 333, 100, dtype, seed=8, resets=True)
    d = on(inp, cuda_device)
    r = reset.to(cuda_device)
    ref = gated.gated_scan(**inp, reset=reset)
    h, parts = None, []
    for lo, hi in ((0, 1), (1, 64), (64, 200), (200, 333)):
        cut = {k: (v[:, lo:hi].contiguous() if k != "lam" else v) for k, v in d.items()}
        y, h = lrs.gated_scan_fwd(**cut, reset=r[:, lo:hi].contiguous(), h0=h, return_final_state=True)
        parts.append(y)
    near(torch.cat(parts, 1), ref, tol_state(333, ref), dtype, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_storage_and_another_stream(cuda_device, dtype):
    """Tensors that start one element into their storage, on a side stream."""
    inp, reset, more = case(2, 130, 128, dtype, seed=11, resets=True)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=cuda_device)
        s[1:].copy_(t.reshape(-1))
        return s[1:].view(t.shape)

    ref = gated.gated_scan(**inp, reset=reset, h0=more["h0"])
    d = {k: shifted(v) for k, v in inp.items()}
    y0 = shifted(torch.zeros_like(inp["x"]))
    r, h0, dy = shifted(reset), shifted(more["h0"]), shifted(more["dy"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, saved = lrs.gated_scan_fwd(**d, reset=r, h0=h0, save="8bit", y=y0)
        saved = {k: shifted(v) for k, v in saved.items()}
        g = lrs.gated_scan_bwd(None, None, None, d["lam"], dy, saved, reset=r)
    side.synchronize()
    assert y.data_ptr() == y0.data_ptr()
    near(y, ref, tol_state(130, ref), dtype, "y")
    _, saved2 = lrs.gated_scan_fwd(**on(inp, cuda_device), reset=reset.to(cuda_device),
                                   h0=more["h0"].to(cuda_device), save="8bit")
    for k in saved:
        near(saved[k], saved2[k].double().cpu().numpy(), 1e-4, "f32", k)
    g2 = lrs.gated_scan_bwd(None, None, None, inp["lam"].to(cuda_device), more["dy"].to(cuda_device), saved2,
                            reset=reset.to(cuda_device))
    for k in g:
        near(g[k], g2[k].double().cpu().numpy(), 2e-3, dtype, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,L,ED", [(1, 900, 75), (2, 257, 1537), (1, 2100, 40), (3, 640, 129)])
def test_clusters_and_rows_off_16_bytes(cuda_device, Bs, L, ED, dtype):
    """Long sequences of few channels (a cluster's blocks share the time axis)
    whose rows start anywhere, with resets, states and 8-bit checkpoints."""
    inp, reset, more = case(Bs, L, ED, dtype, seed=L + 3 * ED, resets=True)
    _, _, saved = check_fwd(inp, reset, more["h0"], dtype, cuda_device, save="8bit")
    values = {}
    for k, q in (("x", "x"), ("gate_r", "r"), ("gate_i", "i")):
        rq, rs = gated.ckpt8(inp[k])
        assert np.array_equal(saved[q + "_q"].cpu().numpy(), rq)
        assert np.array_equal(saved[q + "_s"].cpu().numpy(), rs)
        values[k] = gated.ckpt8_values(rq, rs)
    check_bwd(inp, reset, more, dtype, cuda_device, saved, values)
    check_bwd(inp, reset, more, dtype, cuda_device, {"states": saved["states"]})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,L,ED", [(16, 130, 2560), (20, 150, 1985), (9, 200, 5001)])
def test_more_channels_than_fit_at_a_time(cuda_device, Bs, L, ED, dtype):
    """More than a round of blocks: the last sequences get clusters of their
    own size, in a second launch."""
    inp, reset, more = case(Bs, L, ED, dtype, seed=Bs + ED, resets=True)
    y, hf, saved = check_fwd(inp, reset, more["h0"], dtype, cuda_device, save="8bit")
    y2, hf2, _ = check_fwd(inp, reset, more["h0"], dtype, cuda_device)
    assert torch.equal(y, y2) and torch.equal(hf, hf2)
    values = {}
    for k, q in (("x", "x"), ("gate_r", "r"), ("gate_i", "i")):
        rq, rs = gated.ckpt8(inp[k])
        assert np.array_equal(saved[q + "_q"].cpu().numpy(), rq)
        assert np.array_equal(saved[q + "_s"].cpu().numpy(), rs)
        values[k] = gated.ckpt8_values(rq, rs)
    check_bwd(inp, reset, more, dtype, cuda_device, saved, values)
    check_bwd(inp, reset, more, dtype, cuda_device, {"states": saved["states"]})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,ED", [(70, 128), (700, 64)])
def test_fast_decays(cuda_device, L, ED, dtype):
    """Decays from almost 1 to below 2^-100 in one block of channels."""
    inp, reset, more = case(2, L, ED, dtype, seed=L, resets=True)
    inp["lam"] = torch.linspace(-9.0, 9.0, ED)[torch.randperm(ED, generator=torch.Generator().manual_seed(1))]
    _, _, saved = check_fwd(inp, reset, more["h0"], dtype, cuda_device)
    check_bwd(inp, reset, more, dtype, cuda_device, saved)


def test_y_does_not_depend_on_what_is_kept(cuda_device):
    for Bs, L, ED in ((2, 700, 96), (1, 3000, 64), (2, 500, 72)):
        inp, reset, _ = case(Bs, L, ED, "bf16", seed=L)
        d = on(inp, cuda_device)
        y = lrs.gated_scan_fwd(**d)
        assert torch.equal(y, lrs.gated_scan_fwd(**d, save="states")[0])
        assert torch.equal(y, lrs.gated_scan_fwd(**d, save="8bit")[0])


def test_calls_in_a_cuda_graph(cuda_device):
    """A token step and a forward-backward pair, captured once and replayed on
    new values."""
    inp, _, more = case(3, 200, 128, "bf16", seed=31)
    d = on(inp, cuda_device)
    dy = more["dy"].to(cuda_device)
    tok = {k: v[:, 0].contiguous() if k != "lam" else v for k, v in d.items()}
    states = torch.zeros(4, 128, device=cuda_device)
    pages = torch.tensor([2, -1, 0], dtype=torch.int32, device=cuda_device)

    def work():
        y, saved = lrs.gated_scan_fwd(**d, save="8bit")
        g = lrs.gated_scan_bwd(None, None, None, d["lam"], dy, saved)
        return [y, *g.values(), lrs.gated_scan_step(**tok, states=states, pages=pages)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    d["x"].mul_(0.5)
    tok["x"].mul_(2.0)
    states.fill_(1.0)
    graph.replay()
    got = [t.clone() for t in out]
    states.fill_(1.0)
    for a, b in zip(got, work()):
        assert torch.equal(a, b)


def test_what_follows_a_second_launch(cuda_device):
    """Work behind a pass of two launches sees both, on a stream and in a
    graph: copies queued right after it, and the next pass on its results."""
    inp, _, more = case(16, 130, 2560, "bf16", seed=37)
    d = on(inp, cuda_device)
    dy = more["dy"].to(cuda_device)

    def work():
        y, saved = lrs.gated_scan_fwd(**d, save="states")
        copies = [y.clone()]
        g = lrs.gated_scan_bwd(d["x"], d["gate_r"], d["gate_i"], d["lam"], dy, saved)
        copies += [v.clone() for v in g.values()]
        y2 = lrs.gated_scan_fwd(g["dx"], g["dgate_r"], g["dgate_i"], d["lam"])
        return copies + [y2, y, *g.values()]

    first = work()
    torch.cuda.synchronize()
    for a, b in zip(first[:6], first[7:]):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for a, b in zip(out, first):
            assert torch.equal(a, b)


def test_repeated_calls_are_bitwise_equal(cuda_device):
    inp, reset, more = case(3, 700, 320, "bf16", seed=13, resets=True)
    d, r = on(inp, cuda_device), reset.to(cuda_device)
    first = None
    for _ in range(5):
        y, hf, saved = lrs.gated_scan_fwd(**d, reset=r, return_final_state=True, save="8bit")
        g = lrs.gated_scan_bwd(None, None, None, d["lam"], more["dy"].to(cuda_device), saved, reset=r)
        got = [y, hf, *saved.values(), *g.values()]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_more_than_2_to_31_elements(cuda_device):
    """The tail of a sequence of 2^31 + elements, after a reset, against the
    same steps alone."""
    L, ED = 1_060_000, 2048
    x = torch.empty(1, L, ED, dtype=torch.bfloat16, device=cuda_device)
    x[:, :4096] = 0
    gates = torch.zeros_like(x)
    x.zero_()
    tail = 150
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    x[:, -tail:] = torch.randn(1, tail, ED, generator=gen, device=cuda_device).to(torch.bfloat16)
    gates[:, -tail:] = torch.randn(1, tail, ED, generator=gen, device=cuda_device).to(torch.bfloat16)
    lam = torch.full((ED,), -4.0, device=cuda_device)
    reset = torch.zeros(1, L, dtype=torch.uint8, device=cuda_device)
    reset[:, -tail] = 1
    y, hf, saved = lrs.gated_scan_fwd(x, gates, gates, lam, reset=reset, return_final_state=True, save="8bit")
    cut = [t[:, -tail:].contiguous() for t in (x, gates, gates)]
    ref = gated.gated_scan(*[t.cpu() for t in cut], lam.cpu(), reset=reset[:, -tail:].cpu())
    tol = tol_state(tail, ref)
    near(y[:, -tail:], ref, tol, "bf16", "y")
    near(hf, ref[:, -1], tol, "f32", "h_final")
    assert not y[:, :-tail].any()
    rq, rs = gated.ckpt8(cut[0])
    assert np.array_equal(saved["x_q"][:, -tail:].cpu().numpy(), rq)
    assert np.array_equal(saved["x_s"][:, -tail:].cpu().numpy(), rs)
    del gates
    dy = torch.zeros_like(x)
    dy[:, -tail:] = 1
    g = lrs.gated_scan_bwd(None, None, None, lam, dy, saved, reset=reset)
    assert not g["dx"][:, :-tail].any() and not g["dh0"].any()
    vals = [gated.ckpt8_values(saved[k + "_q"][:, -tail:].cpu().numpy(), saved[k + "_s"][:, -tail:].cpu().numpy())
            for k in "xri"]
    want = gated.gated_scan_bwd(*vals, lam.cpu(), dy[:, -tail:].cpu(),
                                gated.kept_states(gated.gated_scan(*vals, lam.cpu(), reset=reset[:, -tail:].cpu())),
                                reset=reset[:, -tail:].cpu())
    near(g["dx"][:, -tail:], want["dx"], 2 * (16 + tail) * 2.0 ** -21 * max(1, np.abs(want["dx"]).max()), "bf16", "dx")


# ---- one token ------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Bs,ED", [(1, 1), (3, 63), (4, 64), (17, 1536), (300, 130)])
def test_step(cuda_device, Bs, ED, dtype):
    inp, _, more = case(Bs, 1, ED, dtype, seed=Bs + ED)
    n = Bs + 5
    gen = torch.Generator().manual_seed(Bs)
    pool = torch.randn(n, ED, generator=gen)
    pages = torch.randperm(n, generator=gen)[:Bs].to(torch.int32)
    pages[Bs // 2:Bs // 2 + 1] = -1 if ED % 2 else n      # an idle row
    live = ((pages >= 0) & (pages < n)).numpy()
    d = {k: (v[:, 0].contiguous() if k != "lam" else v).to(cuda_device) for k, v in inp.items()}
    states = pool.to(cuda_device)
    y = lrs.gated_scan_step(**d, states=states, pages=pages.to(cuda_device))
    h0 = torch.zeros(Bs, ED)
    h0[live] = pool[pages[live].long()]
    ref = gated.gated_scan(**inp, h0=h0)[:, 0]
    want = pool.double().numpy()
    for b in range(Bs):
        if live[b]:
            want[pages[b]] = ref[b]
        else:
            ref[b] = 0
    near(y, ref, tol_state(1, ref), dtype, "y")
    near(states, want, tol_state(1, want), "f32", "states")
    # without a page list, row b is page b
    states = pool.to(cuda_device)
    y = lrs.gated_scan_step(**d, states=states)
    ref = gated.gated_scan(**inp, h0=pool[:Bs])[:, 0]
    near(y, ref, tol_state(1, ref), dtype, "y, no list")
    assert torch.equal(states[Bs:].cpu(), pool[Bs:])
    near(states[:Bs], ref, tol_state(1, ref), "f32", "states, no list")


def test_steps_follow_the_scan(cuda_device):
    """Tokens one after the other give the scan's outputs."""
    inp, _, _ = case(2, 20, 100, "f32", seed=21)
    d = on(inp, cuda_device)
    y = lrs.gated_scan_fwd(**d)
    states = torch.zeros(2, 100, device=cuda_device)
    got = [lrs.gated_scan_step(d["x"][:, t].contiguous(), d["gate_r"][:, t].contiguous(),
                               d["gate_i"][:, t].contiguous(), d["lam"], states) for t in range(20)]
    ref = gated.gated_scan(**inp)
    near(torch.stack(got, 1), ref, tol_state(20, ref), "f32", "steps")
    near(y, ref, tol_state(20, ref), "f32", "scan")
