"""Cases of the operators around the gated linear recurrence: the recurrence
itself (forward, backward, single-token step), its 8-bit activation
checkpoints, and the pages that hold its states while serving.

Every case computes either the plain form (elementary torch operations in 32
bits) or, where ``own`` is true, the calls a user makes of
linear_recurrence_ssm_gb300.  Sizes are the repository's own channel counts
(64, 1536, 2560, 32 heads of 64 x 128 states) and lengths, and odd ones.
"""
import math

import torch

own = False

BLOCK = 64      # steps between kept states, and columns that share an 8-bit scale
C_GATE = 8.0

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----------------------------------------------------------------------------
def listed():
    return [
        # a short prompt of one request before its first generated token: latency
        dict(name="fwd_short_prompt", op="fwd", Bs=1, L=45, ED=1536, dtype="bf16", reset=False,
             h0=False, final=True, states=False),
        # a training step's forward pass at the library's benchmark shape, keeping what the backward needs
        dict(name="fwd_train", op="fwd", Bs=8, L=2048, ED=1536, dtype="bf16", reset=False,
             h0=False, final=False, states=True),
        # its backward pass
        dict(name="bwd_train", op="bwd", Bs=8, L=2048, ED=1536, dtype="bf16", reset=False,
             dh_final=False),
        # one very long sequence of packed documents, continued from an earlier part
        dict(name="fwd_long_packed", op="fwd", Bs=1, L=65536, ED=2560, dtype="bf16", reset=True,
             h0=True, final=True, states=False),
        # fp32 gradients of packed documents at odd sizes, the sequence continued in a later part
        dict(name="bwd_f32_odd", op="bwd", Bs=3, L=1001, ED=1537, dtype="f32", reset=True,
             dh_final=True),
        # one generated token for each of many requests, some rows of the batch idle
        dict(name="step_batch", op="step", Bs=256, ED=2560, pages=512, dtype="bf16"),
        # a training step with 8-bit checkpoints: forward, then backward from the checkpoint
        dict(name="ckpt8_train", op="ckpt8_train", Bs=16, L=1000, ED=2560, dtype="bf16", reset=False),
        # the same for a small fine-tuning batch of ragged length, packed
        dict(name="ckpt8_train_small", op="ckpt8_train", Bs=2, L=333, ED=200, dtype="bf16", reset=True),
        # another layer's activations kept in 8 bits between its forward and backward pass
        dict(name="ckpt8_keep", op="ckpt8_keep", rows=16384, cols=2048, dtype="bf16"),
        # a beam search step of one request: some beams dropped, others continued twice
        dict(name="pages_beam", op="fork", layers=1, pages=64, elems=1536, n=3, drop=3),
        # many requests that start from the same cached prefixes, full matrix states of several layers
        dict(name="pages_fork_large", op="fork", layers=4, pages=256, elems=262144, n=100, drop=60),
        # the pool made dense again after many requests have ended
        dict(name="pages_compact", op="compact", layers=24, pages=2048, elems=2560, live=1000),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "ckpt8_train", "ckpt8_train", "ckpt8_keep",
                     "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("fwd", "bwd", "ckpt8_train"):
        ED = rng.choice([64, 200, 1536, 2560, _spread(rng, 33, 5000), _spread(rng, 33, 5000)])
        Bs = _spread(rng, 1, 32)
        most = 60_000_000 if op == "fwd" else 30_000_000
        L = _spread(rng, 1, max(1, min(50_000, most // (Bs * ED))))
        case = dict(op=op, Bs=Bs, L=L, ED=ED, dtype=dtype, reset=yes())
        if op == "fwd":
            case.update(h0=yes(), final=yes(), states=yes())
        elif op == "bwd":
            case.update(dh_final=yes())
        return case
    if op == "step":
        Bs = _spread(rng, 1, 1024)
        return dict(op=op, Bs=Bs, ED=rng.choice([1536, 2560, _spread(rng, 33, 8000)]),
                    pages=Bs + _spread(rng, 1, 500), dtype=dtype)
    if op == "ckpt8_keep":
        cols = rng.choice([1536, 2560, _spread(rng, 3, 9000)])
        return dict(op=op, rows=_spread(rng, 1, 60_000_000 // cols), cols=cols, dtype=dtype)
    layers, pages = _spread(rng, 1, 48), _spread(rng, 8, 2000)
    elems = _spread(rng, 64, max(65, min(262144, 200_000_000 // (layers * pages))))
    if op == "fork":
        return dict(op=op, layers=layers, pages=pages, elems=elems, n=_spread(rng, 1, max(1, pages // 2)),
                    drop=rng.randint(0, pages // 4))
    return dict(op=op, layers=layers, pages=pages, elems=elems, live=rng.randint(1, pages))


def work(case):
    """Each input read once, each output written once; a checkpoint that one
    pass writes and reads back counts once for either."""
    op = case["op"]
    if op in ("fwd", "bwd", "ckpt8_train"):
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["Bs"] * case["L"]
        n = rows * case["ED"]
        states = 4 * case["Bs"] * -(-case["L"] // BLOCK) * case["ED"]
        ends = 4 * case["Bs"] * case["ED"]
        resets = rows if case["reset"] else 0
        if op == "fwd":
            b = 4 * e * n + resets + ends * (case["h0"] + case["final"]) + states * case["states"]
            return {"bytes": b + 4 * case["ED"], "flops": 22 * n}
        if op == "bwd":
            b = 7 * e * n + resets + states + ends * (1 + case["dh_final"])
            return {"bytes": b + 8 * case["ED"], "flops": 45 * n}
        kept = 3 * (n + 4 * rows * -(-case["ED"] // BLOCK))
        b = 8 * e * n + 2 * kept + 2 * states + 2 * resets + ends
        return {"bytes": b + 12 * case["ED"], "flops": 70 * n}
    if op == "step":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["Bs"] * (case["ED"] * (4 * e + 8) + 4) + 4 * case["ED"],
                "flops": 22 * case["Bs"] * case["ED"]}
    if op == "ckpt8_keep":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * e * n + 2 * n + 8 * case["rows"] * -(-case["cols"] // BLOCK), "flops": 4 * n}
    moved = case["n"] if op == "fork" else _moves(case["pages"], case["live"])
    return {"bytes": 2 * moved * case["layers"] * case["elems"] * 4 + 2 * case["pages"], "flops": 0}


def _moves(pages, live):
    """Pages that a compaction of `live` randomly placed pages moves, on average."""
    return live * (pages - live) / pages


# ---- inputs ---------------------------------------------------------------------------
def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    t = _TYPES[case.get("dtype", "f32")]

    def normal(*shape, to=t):
        return torch.randn(*shape, generator=g, device=dev).to(to)

    s = dict(case)
    if op in ("fwd", "bwd", "ckpt8_train", "step"):
        # decays exp(-c softplus(lam)) spread over 0.9 .. 0.999, as such layers are initialised
        a = 0.9 + 0.099 * torch.rand(case["ED"], generator=g, device=dev)
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / C_GATE))
    if op == "step":
        Bs, ED = case["Bs"], case["ED"]
        s["x"], s["r"], s["i"] = (normal(Bs, ED) for _ in range(3))
        s["pool"] = normal(case["pages"], ED, to=torch.float32)
        at = torch.randperm(case["pages"], generator=g, device=dev)[:Bs].to(torch.int32)
        s["at"] = torch.where(torch.rand(Bs, generator=g, device=dev) < 0.05, -1, at).to(torch.int32)
    elif op in ("fwd", "bwd", "ckpt8_train"):
        Bs, L, ED = case["Bs"], case["L"], case["ED"]
        s["x"], s["r"], s["i"] = (normal(Bs, L, ED) for _ in range(3))
        # a document ends every few hundred tokens
        s["reset_at"] = (torch.rand(Bs, L, generator=g, device=dev) < 1 / 300).to(torch.uint8) \
            if case["reset"] else None
        if op != "fwd":
            s["dy"] = normal(Bs, L, ED)
        s["start"] = normal(Bs, ED, to=torch.float32) if case.get("h0") else None
        s["dend"] = normal(Bs, ED, to=torch.float32) if case.get("dh_final") else None
    elif op == "ckpt8_keep":
        # activations: most channels of one size, a few much larger
        big = torch.exp(torch.randn(case["cols"], generator=g, device=dev))
        s["x"] = (torch.randn(case["rows"], case["cols"], generator=g, device=dev) * big).to(t)
    else:
        s["pool"] = normal(case["layers"], case["pages"], case["elems"], to=torch.float32)
        order = torch.randperm(case["pages"], generator=g, device=dev).to(torch.int32)
        used = torch.zeros(case["pages"], dtype=torch.uint8, device=dev)
        if op == "fork":
            # a pool two thirds full; `drop` of its pages end now, the requests continue others (one starts anew)
            live = max(1, min(case["pages"] * 2 // 3, case["pages"] - case["n"] + case["drop"]))
            used[order[:live].long()] = 1
            s["ended"] = order[:min(case["drop"], live - 1)].contiguous()
            kept = order[min(case["drop"], live - 1):live]
            pick = torch.randint(0, kept.numel(), (case["n"],), generator=g, device=dev)
            s["src"] = kept[pick].contiguous()
            s["src"][-1] = -1
        else:
            used[order[:case["live"]].long()] = 1
            s["at"] = order[:case["live"]].contiguous()
        s["used"] = used
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "bwd":   # the forward pass has kept its states
        a, b, _ = _gates(s["x"], s["r"], s["i"], s["lam"], s["reset_at"])
        s["kept"] = _entering(_scan(a, b), None)
    return s


# ---- plain forms ----------------------------------------------------------------------
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def _gates(x, r, i, lam, reset):
    """(a, b, parts of the gradients) of h_t = a_t h_{t-1} + b_t in 32 bits."""
    x, sr, si = x.float(), _sigmoid(r.float()), _sigmoid(i.float())
    la = -C_GATE * _softplus(lam) * sr
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    if reset is not None:
        at = reset.bool().unsqueeze(-1)
        a, m, la = a.masked_fill(at, 0.0), m.masked_fill(at, 1.0), la.masked_fill(at, 0.0)
    return a, m * si * x, (x, sr, si, la, m)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from 0, by doubling."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat((b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])), 1)
        a = torch.cat((a[:, :k], a[:, k:] * a[:, :-k]), 1)
        k *= 2
    return b


def _entering(h, h0):
    """The states that enter the blocks of 64 steps: (Bs, blocks, ED)."""
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0.unsqueeze(1)
    return torch.cat((first, h[:, BLOCK - 1:-1:BLOCK]), 1)


def _in_blocks(v, fill):
    pad = -v.shape[1] % BLOCK
    if pad:
        v = torch.cat((v, v.new_full((v.shape[0], pad, v.shape[2]), fill)), 1)
    return v.reshape(-1, BLOCK, v.shape[2])


def _plain_fwd(x, r, i, lam, reset, h0):
    a, b, _ = _gates(x, r, i, lam, reset)
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    return _scan(a, b)


def _plain_bwd(x, r, i, lam, reset, dy, kept, dend, to):
    a, b, (x, sr, si, la, m) = _gates(x, r, i, lam, reset)
    Bs, L, ED = a.shape
    # the state before each step, from the kept states
    ab, bb = _in_blocks(a, 1.0), _in_blocks(b, 0.0)
    start = kept.reshape(-1, ED)
    bb[:, 0] += ab[:, 0] * start
    before = torch.cat((start.unsqueeze(1), _scan(ab, bb)[:, :-1]), 1).reshape(Bs, -1, ED)[:, :L]
    # g_t = dy_t + a_{t+1} g_{t+1}
    d = dy.float()
    if dend is not None:
        d = torch.cat((d[:, :-1], d[:, -1:] + dend.unsqueeze(1)), 1)
    after = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    g = _scan(after.flip(1), d.flip(1)).flip(1)
    G = la * g * (a * before - a * a / m.clamp(min=1e-30) * si * x)
    gm = g * m * si
    dlam = G.sum((0, 1)) * _sigmoid(lam) / _softplus(lam)
    return {"dx": gm.to(to), "dgate_r": (G * (1 - sr)).to(to), "dgate_i": (gm * x * (1 - si)).to(to),
            "dlam": dlam, "dh0": a[:, 0] * g[:, 0]}


def _in_groups(x):
    v = x.reshape(-1, x.shape[-1]).float()
    pad = -v.shape[1] % BLOCK
    if pad:
        v = torch.cat((v, v.new_zeros(v.shape[0], pad)), 1)
    return v.reshape(v.shape[0], -1, BLOCK)


def _through_8bit(x):
    """The values that x's 8-bit checkpoint stands for, in 32 bits."""
    v = _in_groups(x)
    top = v.abs().amax(-1, keepdim=True)
    none = top < 2.0 ** -100
    inv = torch.div(torch.full_like(top, 127.0), top).masked_fill(none, 0.0)
    scale = (top * torch.tensor(1 / 127, dtype=torch.float32, device=x.device)).masked_fill(none, 0.0)
    return (torch.round(v * inv) * scale).flatten(1)[:, :x.shape[-1]].reshape(x.shape)


def _plain(s):
    op = s["op"]
    if op == "fwd":
        h = _plain_fwd(s["x"], s["r"], s["i"], s["lam"], s["reset_at"], s["start"])
        out = {"y": h.to(s["x"].dtype)}
        if s["final"]:
            out["h_final"] = h[:, -1]
        if s["states"]:
            out["states"] = _entering(h, s["start"])
        return out
    if op == "bwd":
        return _plain_bwd(s["x"], s["r"], s["i"], s["lam"], s["reset_at"], s["dy"], s["kept"],
                          s["dend"], s["x"].dtype)
    if op == "ckpt8_train":
        h = _plain_fwd(s["x"], s["r"], s["i"], s["lam"], s["reset_at"], None)
        out = _plain_bwd(_through_8bit(s["x"]), _through_8bit(s["r"]), _through_8bit(s["i"]), s["lam"],
                         s["reset_at"], s["dy"], _entering(h, None), None, s["x"].dtype)
        out["y"] = h.to(s["x"].dtype)
        return out
    if op == "step":
        a, b, _ = _gates(s["x"], s["r"], s["i"], s["lam"], None)
        idle = (s["at"] < 0).unsqueeze(-1)
        # an idle row goes through a row of its own below the pool
        at = torch.where(s["at"] < 0, s["pages"], s["at"]).long()
        whole = torch.cat((s["pool"], s["pool"].new_zeros(1, s["ED"])))
        h = a * whole[at] + b
        whole[at] = h
        s["pool"].copy_(whole[:-1])
        return {"y": h.masked_fill(idle, 0.0).to(s["x"].dtype), "states": s["pool"]}
    if op == "ckpt8_keep":
        return _through_8bit(s["x"]).to(s["x"].dtype)
    pool, used = s["pool"], s["used"].clone()
    if op == "fork":
        used[s["ended"].long()] = 0
        src = s["src"].long()
        free = torch.nonzero(used == 0).flatten()
        n = min(src.numel(), free.numel())
        dst = torch.full_like(s["src"], -1)
        dst[:n] = free[:n].to(torch.int32)
        pool[:, free[:n]] = pool[:, src[:n].clamp(min=0)] * (src[:n] >= 0).view(1, -1, 1)
        used[free[:n]] = 1
        return {"pool": pool, "used": used, "dst": dst}
    live = int(s["at"].numel())
    page = torch.arange(s["pages"], device=used.device)
    hole, mover = page[(used == 0) & (page < live)], page[(used != 0) & (page >= live)]
    pool[:, hole] = pool[:, mover]
    moved = torch.where(used != 0, page, -1)
    moved[mover] = hole
    return {"pool": pool, "used": (page < live).to(torch.uint8), "at": moved[s["at"].long()].to(torch.int32)}


# ---- one pass -------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import linear_recurrence_ssm_gb300 as lrs
    op = s["op"]
    if op == "fwd":
        got = lrs.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], c=C_GATE, reset=s["reset_at"],
                                 h0=s["start"], return_final_state=s["final"],
                                 save="states" if s["states"] else None)
        got = list(got) if isinstance(got, tuple) else [got]
        out = {"y": got.pop(0)}
        if s["final"]:
            out["h_final"] = got.pop(0)
        if s["states"]:
            out["states"] = got.pop(0)["states"]
        return out
    if op == "bwd":
        return lrs.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], {"states": s["kept"]},
                                  c=C_GATE, reset=s["reset_at"], dh_final=s["dend"])
    if op == "ckpt8_train":
        y, saved = lrs.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], c=C_GATE, reset=s["reset_at"],
                                      save="8bit")
        out = lrs.gated_scan_bwd(None, None, None, s["lam"], s["dy"], saved, c=C_GATE,
                                 reset=s["reset_at"])
        out["y"] = y
        return out
    if op == "step":
        y = lrs.gated_scan_step(s["x"], s["r"], s["i"], s["lam"], s["pool"], s["at"], c=C_GATE)
        return {"y": y, "states": s["pool"]}
    if op == "ckpt8_keep":
        q, scale = lrs.ckpt8_save(s["x"])
        return lrs.ckpt8_load(q, scale, s["x"].dtype)
    used = s["used"].clone()
    if op == "fork":
        lrs.state_pages_free(used, s["ended"])
        dst = lrs.state_pages_fork(s["pool"], used, s["src"], page_dim=1)
        return {"pool": s["pool"], "used": used, "dst": dst}
    at = s["at"].clone()
    lrs.state_pages_compact(s["pool"], used, at, page_dim=1)
    return {"pool": s["pool"], "used": used, "at": at}


# ---- 64 bits --------------------------------------------------------------------------
def _exact_gate(x, r, i, lam, reset):
    """One value or many of the recurrence's coefficients, from their definition."""
    f = torch.float64
    sr, si = 1 / (1 + torch.exp(-r.to(f))), 1 / (1 + torch.exp(-i.to(f)))
    la = -C_GATE * torch.log1p(torch.exp(lam.to(f))) * sr
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    if reset is not None:
        keep = (reset == 0).to(f)[..., None]
        a, m, la = a * keep, m * keep + (1 - keep), la * keep
    return x.to(f), sr, si, la, a, m


def _exact_states(x, si, a, m, start):
    h = torch.empty_like(a)
    last = torch.zeros_like(a[:, 0]) if start is None else start.double()
    for t in range(a.shape[1]):
        last = a[:, t] * last + m[:, t] * si[:, t] * x[:, t]
        h[:, t] = last
    return h


def _exact_grads(x, r, i, lam, reset, dy, kept, dend):
    x, sr, si, la, a, m = _exact_gate(x, r, i, lam, reset)
    Bs, L, ED = a.shape
    before = torch.empty_like(a)
    for j in range(BLOCK):      # step j of every block
        n = before[:, j::BLOCK].shape[1]
        if not n:
            break
        if j == 0:
            last = kept[:, :n].double()
        else:
            at = slice(j - 1, L - 1, BLOCK)     # the steps before those
            last = a[:, at] * before[:, at] + m[:, at] * si[:, at] * x[:, at]
        before[:, j::BLOCK] = last
    g = torch.empty_like(a)
    u = torch.zeros_like(a[:, 0]) if dend is None else dend.double()
    for t in range(L - 1, -1, -1):
        g[:, t] = dy[:, t].double() + u
        u = a[:, t] * g[:, t]
    dsi = g * m * x
    dla = g * (a * before - a * a * si * x / m)
    sp = torch.log1p(torch.exp(lam.double()))
    dsr = dla * (-C_GATE * sp)
    if reset is not None:
        dsr = dsr * (reset == 0).double()[..., None]
        dla = dla * (reset == 0).double()[..., None]
    dlam = (dla * sr).sum((0, 1)) * -C_GATE / (1 + torch.exp(-lam.double()))
    return {"dx": g * m * si, "dgate_r": dsr * sr * (1 - sr), "dgate_i": dsi * si * (1 - si),
            "dlam": dlam, "dh0": u}


def _exact_8bit(x):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[-1], BLOCK):
        v = x[..., k:k + BLOCK].double()
        top = v.abs().amax(-1, keepdim=True)
        step = top / 127
        out[..., k:k + BLOCK] = torch.where(top < 2.0 ** -100, 0.0, torch.round(v / step) * step)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fwd":
        x, _, si, _, a, m = _exact_gate(s["x"], s["r"], s["i"], s["lam"], s["reset_at"])
        h = _exact_states(x, si, a, m, s["start"])
        out = {"y": h}
        if case["final"]:
            out["h_final"] = h[:, -1]
        if case["states"]:
            first = torch.zeros_like(h[:, :1]) if s["start"] is None else s["start"].double()[:, None]
            out["states"] = torch.cat([first] + [h[:, t - 1:t] for t in range(BLOCK, case["L"], BLOCK)], 1)
        return out
    if op == "bwd":
        return _exact_grads(s["x"], s["r"], s["i"], s["lam"], s["reset_at"], s["dy"], s["kept"], s["dend"])
    if op == "ckpt8_train":
        x, _, si, _, a, m = _exact_gate(s["x"], s["r"], s["i"], s["lam"], s["reset_at"])
        h = _exact_states(x, si, a, m, None)
        kept = torch.stack([torch.zeros_like(h[:, 0])] + [h[:, t - 1] for t in range(BLOCK, case["L"], BLOCK)], 1)
        out = _exact_grads(_exact_8bit(s["x"]), _exact_8bit(s["r"]), _exact_8bit(s["i"]), s["lam"],
                           s["reset_at"], s["dy"], kept, None)
        out["y"] = h
        return out
    if op == "step":
        x, _, si, _, a, m = _exact_gate(s["x"], s["r"], s["i"], s["lam"], None)
        pool = s["pool"].double()
        y = torch.zeros_like(x)
        for b, p in enumerate(s["at"].tolist()):
            if p >= 0:
                y[b] = a[b] * pool[p] + m[b] * si[b] * x[b]
                pool[p] = y[b]
        return {"y": y, "states": pool}
    if op == "ckpt8_keep":
        return _exact_8bit(s["x"])
    if case["layers"] * case["pages"] * case["elems"] > 400_000_000:
        return None
    pool, used = s["pool"].double(), s["used"].tolist()
    if op == "fork":
        for p in s["ended"].tolist():
            used[p] = 0
        dst = []
        for p in s["src"].tolist():
            q = used.index(0) if 0 in used else -1
            dst.append(q)
            if q >= 0:
                used[q] = 1
                pool[:, q] = s["pool"][:, p].double() if p >= 0 else 0.0
        return {"pool": pool, "used": None, "dst": None}
    live = sum(used)
    moves = [p for p in range(case["pages"]) if used[p] and p >= live]
    for p in range(live):
        if not used[p]:
            q = moves.pop(0)
            pool[:, p] = pool[:, q].clone()
    return {"pool": pool, "used": None, "at": None}
