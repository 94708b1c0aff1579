"""Cases of the gated delta rule (forward, training pass, single-token step on
state pages) and of the root-mean-square norm around it (with the residual's
addition, an 8-bit output and gradients).

Every case computes either the plain form (elementary torch operations in 32
bits) or, where ``own`` is true, the calls a user makes of
linear_recurrence_ssm_gb300.  Sizes are the repository's own heads (32 of
64 x 128 states, 8 of 64 x 64), widths (1536, 2048, 2560) and lengths, and odd
ones.
"""
import math

import torch

own = False

BLOCK = 64      # steps that the plain form takes at once, and columns that share an 8-bit scale
EPS = 1e-6

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----------------------------------------------------------------------------
# delta rule: n sequences; packed: of different lengths behind one another, L tokens in all, else n of L tokens
def listed():
    return [
        # a short prompt of one request before its first generated token: latency
        dict(name="delta_short_prompt", op="delta_fwd", n=1, L=45, packed=False, G=16, H=32, K=128, V=64,
             dtype="bf16", h0=False, final=True),
        # the prompts of several requests in one pass, each continuing a state of its own
        dict(name="delta_prompts_packed", op="delta_fwd", n=11, L=16384, packed=True, G=16, H=32, K=128, V=64,
             dtype="bf16", h0=True, final=True),
        # one very long prompt, few heads
        dict(name="delta_long_prompt", op="delta_fwd", n=1, L=65536, packed=False, G=8, H=8, K=128, V=128,
             dtype="bf16", h0=False, final=True),
        # a training step at the library's benchmark shape of matrix states
        dict(name="delta_train", op="delta_train", n=4, L=4096, packed=False, G=32, H=32, K=128, V=64,
             dtype="bf16", h0=False, final=False),
        # a small fine-tuning batch of packed documents that continue earlier parts and are continued
        dict(name="delta_train_packed", op="delta_train", n=7, L=1999, packed=True, G=4, H=8, K=64, V=64,
             dtype="bf16", h0=True, final=True),
        # fp32 at odd sizes
        dict(name="delta_train_f32_odd", op="delta_train", n=3, L=333, packed=False, G=5, H=5, K=96, V=40,
             dtype="f32", h0=False, final=True),
        # one generated token for each of many requests, some rows of the batch idle
        dict(name="delta_step_batch", op="delta_step", Bs=256, pages=512, G=16, H=32, K=128, V=64, dtype="bf16"),
        # one generated token of one request
        dict(name="delta_step_one", op="delta_step", Bs=1, pages=16, G=8, H=8, K=64, V=64, dtype="bf16"),
        # the norm before a layer, its output kept in 8 bits, the residual carried on
        dict(name="norm_8bit", op="norm_fwd", rows=16384, cols=2048, dtype="bf16", residual=True, out="8bit"),
        # the same norm for the tokens of one generation step
        dict(name="norm_step", op="norm_fwd", rows=64, cols=2560, dtype="bf16", residual=True, out="same"),
        # a training step's norm: forward, then gradients, the residual's gradient joined
        dict(name="norm_train", op="norm_train", rows=16384, cols=2560, dtype="bf16", residual=True),
        # the norm of single heads in fp32, odd rows
        dict(name="norm_train_heads_f32", op="norm_train", rows=100001, cols=64, dtype="f32", residual=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_train", "delta_train", "delta_step", "norm_fwd", "norm_train"])
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("delta_fwd", "delta_train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        K, V = rng.choice([(128, 64), (128, 128), (64, 64), (64, 128), (96, 40), (16, 16),
                           (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))])
        G = rng.choice([1, 2, 4, 5, 8, 16])
        H = G * rng.choice([1, 1, 2, 3])
        n = _spread(rng, 1, 16)
        packed = yes()
        most = (262144 if op == "delta_fwd" else 131072) // (4 if dtype == "f32" else 1)
        L = _spread(rng, 1, max(1, min(16384, most // (H * n))))
        return dict(op=op, n=n, L=L * n if packed else L, packed=packed, G=G, H=H, K=K, V=V, dtype=dtype,
                    h0=yes(), final=yes())
    if op == "delta_step":
        K, V = rng.choice([(128, 64), (128, 128), (64, 64), (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))])
        G = rng.choice([1, 4, 8, 16])
        Bs = _spread(rng, 1, 300)
        return dict(op=op, Bs=Bs, pages=Bs + _spread(rng, 1, 200), G=G, H=G * rng.choice([1, 2]), K=K, V=V,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    cols = rng.choice([64, 128, 1536, 2048, 2560, _spread(rng, 33, 9000)])
    rows = _spread(rng, 1, 33_000_000 // cols)
    if op == "norm_fwd" and yes():
        return dict(op=op, rows=rows, cols=cols, dtype="bf16", residual=yes(), out="8bit")
    case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=yes())
    return dict(case, out="same") if op == "norm_fwd" else case


def work(case):
    """Each input read once, each output written once; what one pass keeps for
    its gradients is not counted."""
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("delta_fwd", "delta_train"):
        t = case["L"] * (1 if case["packed"] else case["n"])
        G, H, K, V = case["G"], case["H"], case["K"], case["V"]
        qk, v, gates, state = 2 * t * G * K, t * H * V, 2 * t * H, 4 * case["n"] * H * K * V
        b = e * (qk + 2 * v + gates) + state * (case["h0"] + case["final"])
        step = H * t * K * V
        if op == "delta_fwd":
            return {"bytes": b, "flops": 6 * step}
        b += e * (2 * qk + 2 * v + 2 * gates) + state * (case["h0"] + case["final"])
        return {"bytes": b, "flops": 20 * step}
    if op == "delta_step":
        G, H, K, V = case["G"], case["H"], case["K"], case["V"]
        return {"bytes": case["Bs"] * (e * (2 * G * K + 2 * H * V + 2 * H) + 8 * H * K * V + 4),
                "flops": 7 * case["Bs"] * H * K * V}
    n = case["rows"] * case["cols"]
    if op == "norm_fwd":
        o = n + 4 * case["rows"] * -(-case["cols"] // BLOCK) if case["out"] == "8bit" else e * n
        return {"bytes": e * n * (3 if case["residual"] else 1) + o + 4 * case["cols"], "flops": 5 * n}
    return {"bytes": e * n * (7 if case["residual"] else 4) + 8 * case["cols"], "flops": 15 * n}


# ---- inputs ---------------------------------------------------------------------------
def _lengths(total, n, seed):
    """n lengths of at least one token that make up `total`, from short to many times as long."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(1.2 * torch.randn(n, generator=g))
    cut = [0] + [min(int(c), total) for c in torch.round(torch.cumsum(w, 0) / w.sum() * total).tolist()]
    cut[-1] = total
    if total >= n:      # every sequence has a token
        for i in range(1, n):
            cut[i] = min(max(cut[i], cut[i - 1] + 1), total - (n - i))
    return [b - a for a, b in zip(cut, cut[1:])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, to=t):
        return torch.randn(*shape, generator=g, device="cuda").to(to)

    s = dict(case)
    op = case["op"]
    if op.startswith("delta"):
        G, H, K, V = case["G"], case["H"], case["K"], case["V"]
        if op == "delta_step":
            rows = (case["Bs"],)
        else:
            rows = (1, case["L"]) if case["packed"] else (case["n"], case["L"])

        def unit():
            """Directions, as a layer's activation and norm leave them; neighbours resemble one another."""
            w = torch.nn.functional.silu(normal(*rows, G, K, to=torch.float32) + 0.3 * normal(1, G, K, to=torch.float32))
            return (w / w.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(t)

        s["q"], s["k"], s["v"] = unit(), unit(), normal(*rows, H, V)
        # decays of a step spread over 0.9 .. 0.999 by head, varied by token
        rate = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(H, generator=g, device="cuda"))
        s["g"] = (-rate * torch.nn.functional.softplus(normal(*rows, H, to=torch.float32) + 0.5)).to(t)
        s["beta"] = torch.sigmoid(normal(*rows, H, to=torch.float32)).to(t)
        if op == "delta_step":
            s["pool"] = 0.1 * normal(case["pages"], H, V, K, to=torch.float32)
            at = torch.randperm(case["pages"], generator=g, device="cuda")[:case["Bs"]].to(torch.int32)
            if case["Bs"] > 1:
                at = torch.where(torch.rand(case["Bs"], generator=g, device="cuda") < 0.05, -1, at).to(torch.int32)
            s["at"] = at
            return s
        s["lengths"] = _lengths(case["L"], case["n"], seed) if case["packed"] else [case["L"]] * case["n"]
        s["offsets"] = None
        if case["packed"]:
            ends = [sum(s["lengths"][:i]) for i in range(case["n"] + 1)]
            s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["start"] = 0.1 * normal(case["n"], H, V, K, to=torch.float32) if case["h0"] else None
        if op == "delta_train":
            s["dy"] = normal(*rows, H, V)
            s["dend"] = normal(case["n"], H, V, K, to=torch.float32) if case["final"] else None
        return s
    rows, cols = case["rows"], case["cols"]
    # activations: most channels of one size, a few much larger
    big = torch.exp(torch.randn(cols, generator=g, device="cuda"))
    s["x"] = (torch.randn(rows, cols, generator=g, device="cuda") * big).to(t)
    s["weight"] = 1.0 + 0.2 * normal(cols, to=torch.float32)
    s["r"] = (torch.randn(rows, cols, generator=g, device="cuda") * big).to(t) if case["residual"] else None
    if op == "norm_train":
        s["dy"] = normal(rows, cols)
        s["ds"] = normal(rows, cols) if case["residual"] else None
    return s


# ---- plain forms ----------------------------------------------------------------------
def _rows_of(s):
    """Where each sequence's tokens lie in the flat batch, padded to whole blocks: (n, Lp) and whether there is one."""
    n, dev = len(s["lengths"]), s["q"].device
    most = max(s["lengths"])
    padded = -(-max(most, 1) // BLOCK) * BLOCK
    length = torch.tensor(s["lengths"], device=dev)
    first = torch.cumsum(length, 0) - length
    at = torch.arange(padded, device=dev)
    there = at < length.view(n, 1)
    return torch.where(there, first.view(n, 1) + at, 0), there


def _inverse(a):
    """(1 + a)^-1 of strictly lower triangular a, by blocks of doubled size."""
    C = a.shape[-1]
    t = torch.eye(C, device=a.device).expand(a.shape)
    at = torch.arange(C, device=a.device)
    w = 1
    while w < C:
        corner = (at.view(C, 1) // w % 2 == 1) & (at.view(1, C) // w == at.view(C, 1) // w - 1)
        t = t - t @ (a * corner) @ t
        w *= 2
    return t


def _passed(M, b):
    """S_c = M_c S_{c-1} + b_c along dimension 2 from 0, by doubling."""
    k = 1
    while k < b.shape[2]:
        b = torch.cat((b[:, :, :k], b[:, :, k:] + M[:, :, k:] @ b[:, :, :-k]), 2)
        M = torch.cat((M[:, :, :k], M[:, :, k:] @ M[:, :, :-k]), 2)
        k *= 2
    return b


def _plain_delta(s, q, k, v, g, beta, start):
    """(y flat, final states) in 32 bits, 64 steps at a time."""
    G, H, K, V = s["G"], s["H"], s["K"], s["V"]
    at, there = _rows_of(s)
    n, Lp = at.shape

    def blocks(w):      # (tokens, heads, ...) -> (n, H, blocks, 64, ...), 0 behind a sequence's end
        w = w[at] * there.view(n, Lp, *(1,) * (w.dim() - 1))
        w = w.repeat_interleave(H // w.shape[2], 2)
        return w.reshape(n, -1, BLOCK, *w.shape[2:]).movedim(3, 1)

    q, k, v = (blocks(w.flatten(0, 1).float()) for w in (q, k, v))
    beta = blocks(beta.flatten(0, 1).float())
    gamma = blocks(g.flatten(0, 1).double()).cumsum(-1)         # 64 bits: differences of these count
    low = torch.tril(torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=q.device))
    D = torch.exp((gamma.unsqueeze(-1) - gamma.unsqueeze(-2)).masked_fill(~low, -math.inf).float())
    Gam, E = torch.exp(gamma.float()), torch.exp((gamma[..., -1:] - gamma).float())
    T = _inverse(torch.tril(k @ k.mT * D, -1) * beta.unsqueeze(-2))
    XV, XK = T @ v, T @ (Gam.unsqueeze(-1) * k)
    kept = (k * (E * beta).unsqueeze(-1)).mT                     # (K, 64)
    M = Gam[..., -1, None, None] * torch.eye(K, device=q.device) - kept @ XK
    b = kept @ XV
    first = torch.zeros(n, H, K, V, device=q.device) if start is None else start.mT
    b = torch.cat((b[:, :, :1] + M[:, :, :1] @ first.unsqueeze(2), b[:, :, 1:]), 2)
    after = _passed(M, b)
    before = torch.cat((first.unsqueeze(2), after[:, :, :-1]), 2)
    U = (XV - XK @ before) * beta.unsqueeze(-1)
    y = (Gam.unsqueeze(-1) * (q @ before) + (q @ k.mT * D) @ U) * K ** -0.5
    y = y.movedim(1, 3).reshape(n, Lp, H, V)
    return y[there], after[:, :, -1].mT     # sequences lie in their order, so rows come out in theirs


def _plain_delta_train(s):
    leaves = [s[w].detach().clone().requires_grad_() for w in ("q", "k", "v", "g", "beta")]
    start = None if s["start"] is None else s["start"].detach().clone().requires_grad_()
    with torch.enable_grad():
        y, end = _plain_delta(s, *leaves, start)
        ends = [(y, s["dy"].flatten(0, 1).float())] + ([(end, s["dend"])] if s["final"] else [])
        wanted = leaves + ([start] if start is not None else [])
        got = torch.autograd.grad([a for a, _ in ends], wanted, [b for _, b in ends])
    out = dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got))
    out["y"] = y.detach().to(s["v"].dtype).view(s["v"].shape)
    if s["final"]:
        out["h_final"] = end.detach().contiguous()
    return out


def _plain_delta_step(s):
    H, K = s["H"], s["K"]
    q, k = (w.float().repeat_interleave(H // s["G"], 1) for w in (s["q"], s["k"]))
    idle = s["at"] < 0
    at = s["at"].clamp(min=0).long()
    old = s["pool"][at] * torch.exp(s["g"].float()).view(-1, H, 1, 1)
    u = s["beta"].float().unsqueeze(-1) * (s["v"].float() - (old * k.unsqueeze(2)).sum(-1))
    new = old + u.unsqueeze(-1) * k.unsqueeze(2)
    y = (new * q.unsqueeze(2)).sum(-1) * K ** -0.5
    s["pool"][torch.where(idle, s["pages"], at)[~idle]] = new[~idle]
    return {"y": y.masked_fill(idle.view(-1, 1, 1), 0.0).to(s["v"].dtype), "states": s["pool"]}


def _through_8bit(x):
    """The values that x's 8-bit form (a scale for 64 columns) stands for, in 32 bits."""
    pad = -x.shape[1] % BLOCK
    v = torch.cat((x, x.new_zeros(x.shape[0], pad)), 1) if pad else x
    v = v.view(x.shape[0], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    none = top < 2.0 ** -100
    inv = torch.div(torch.full_like(top, 127.0), top).masked_fill(none, 0.0)
    scale = (top * torch.tensor(1 / 127, dtype=torch.float32, device=x.device)).masked_fill(none, 0.0)
    return (torch.round(v * inv) * scale).flatten(1)[:, :x.shape[1]]


def _plain_norm(s):
    t = s["x"].dtype
    a = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    rstd = torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS)
    y = a * rstd * s["weight"]
    if s["op"] == "norm_fwd":
        out = {"y": _through_8bit(y).to(t) if s["out"] == "8bit" else y.to(t)}
        if s["r"] is not None:
            out["sum"] = a.to(t)
        return out
    out = {"y": y.to(t)}
    d = s["dy"].float()
    wd = d * s["weight"]
    dx = rstd * (wd - a * rstd * rstd * (wd * a).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
        out["sum"] = a.to(t)
    out["dx"] = dx.to(t)
    out["dweight"] = (d * a * rstd).sum(0)
    return out


def _plain(s):
    op = s["op"]
    if op == "delta_fwd":
        y, end = _plain_delta(s, s["q"], s["k"], s["v"], s["g"], s["beta"], s["start"])
        out = {"y": y.to(s["v"].dtype).view(s["v"].shape)}
        return dict(out, h_final=end.contiguous()) if s["final"] else out
    if op == "delta_train":
        return _plain_delta_train(s)
    if op == "delta_step":
        return _plain_delta_step(s)
    return _plain_norm(s)


# ---- one pass -------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import linear_recurrence_ssm_gb300 as lrs
    op = s["op"]
    if op == "delta_fwd":
        got = lrs.delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], offsets=s["offsets"], h0=s["start"],
                                 return_final_state=s["final"])
        return {"y": got[0], "h_final": got[1]} if s["final"] else {"y": got}
    if op == "delta_train":
        got = lrs.delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], offsets=s["offsets"], h0=s["start"],
                                 return_final_state=s["final"], save="states")
        out = lrs.delta_rule_bwd(s["q"], s["k"], s["g"], s["beta"], s["dy"], got[-1], offsets=s["offsets"],
                                 dh_final=s["dend"], need_dh0=s["h0"])
        out = {name: w for name, w in out.items() if w is not None}
        out["y"] = got[0]
        return dict(out, h_final=got[1]) if s["final"] else out
    if op == "delta_step":
        y = lrs.delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["at"])
        return {"y": y, "states": s["pool"]}
    if op == "norm_fwd":
        if s["out"] == "8bit":
            got = lrs.rms_norm_fwd(s["x"], s["weight"], residual=s["r"], eps=EPS, out="8bit")
            out = {"y": lrs.ckpt8_load(got[0], got[1], s["x"].dtype)}
            return dict(out, sum=got[2]) if s["r"] is not None else out
        got = lrs.rms_norm_fwd(s["x"], s["weight"], residual=s["r"], eps=EPS)
        return {"y": got[0], "sum": got[1]} if s["r"] is not None else {"y": got}
    got = lrs.rms_norm_fwd(s["x"], s["weight"], residual=s["r"], eps=EPS, save=True)
    out = {"y": got[0]}
    if s["r"] is not None:
        out["sum"] = got[1]
    grads = lrs.rms_norm_bwd(s["dy"], s["x"], s["weight"], got[-1], residual=s["r"], ds=s["ds"])
    return dict(out, dx=grads["dx"], dweight=grads["dweight"])


# ---- 64 bits --------------------------------------------------------------------------
def _steps(s):
    """The tokens of all sequences side by side, (longest, n, heads, ...) in 64 bits; behind an end: no decay, no write."""
    longest, n = max(s["lengths"] + [1]), s["n"]

    def apart(w, fill):
        w = w.reshape(-1, *w.shape[2:]).double()
        out = w.new_full((longest, n) + w.shape[1:], fill)
        at = 0
        for i, l in enumerate(s["lengths"]):
            out[:l, i] = w[at:at + l]
            at += l
        return out

    r = s["H"] // s["G"]
    q, k = (apart(s[w], 0.0).repeat_interleave(r, 2) for w in ("q", "k"))
    return q * s["K"] ** -0.5, k, apart(s["v"], 0.0), torch.exp(apart(s["g"], 0.0)), apart(s["beta"], 0.0), apart


def _together(s, w):
    """(longest, n, ...) back in the batch's order."""
    return torch.cat([w[:l, i] for i, l in enumerate(s["lengths"])])


def _one_step(S, k, v, a, b):
    S = S * a[..., None, None]
    x = v - (S @ k.unsqueeze(-1)).squeeze(-1)
    return S + (b.unsqueeze(-1) * x).unsqueeze(-1) * k.unsqueeze(-2), x


def _exact_delta(s, grads):
    q, k, v, a, b, apart = _steps(s)
    T, n, H, V = v.shape
    S = torch.zeros(n, H, V, s["K"], dtype=torch.float64, device=v.device)
    if s["start"] is not None:
        S = s["start"].double().clone()
    y, kept = torch.empty_like(v), []
    for t in range(T):
        if grads and t % 64 == 0:
            kept.append(S)
        S, _ = _one_step(S, k[t], v[t], a[t], b[t])
        y[t] = (S @ q[t].unsqueeze(-1)).squeeze(-1)
    out = {"y": _together(s, y).view(s["v"].shape)}
    if s["final"]:
        out["h_final"] = S
    if not grads:
        return out
    dy = apart(s["dy"], 0.0)
    dq, dk, dv, dg, db = (torch.empty_like(w) for w in (q, k, v, a, b))
    A = torch.zeros_like(S) if s["dend"] is None else s["dend"].double().clone()
    for c in range(len(kept) - 1, -1, -1):
        inside, S = [], kept[c]
        for t in range(64 * c, min(64 * c + 64, T)):
            old = S
            S, x = _one_step(S, k[t], v[t], a[t], b[t])
            inside.append((t, old * a[t][..., None, None], x, S))
        for t, old, x, S in reversed(inside):
            dq[t] = (S.mT @ dy[t].unsqueeze(-1)).squeeze(-1)
            A = A + dy[t].unsqueeze(-1) * q[t].unsqueeze(-2)
            du = (A @ k[t].unsqueeze(-1)).squeeze(-1)
            db[t] = (du * x).sum(-1)
            dx = b[t].unsqueeze(-1) * du
            dk[t] = ((A.mT @ (b[t].unsqueeze(-1) * x).unsqueeze(-1)) - old.mT @ dx.unsqueeze(-1)).squeeze(-1)
            dv[t] = dx
            A = A - dx.unsqueeze(-1) * k[t].unsqueeze(-2)
            dg[t] = (A * old).sum((-2, -1))
            A = A * a[t][..., None, None]
    dq, dk = (w.unflatten(2, (s["G"], -1)).sum(3) for w in (dq * s["K"] ** -0.5, dk))
    for name, w, like in (("dq", dq, "q"), ("dk", dk, "k"), ("dv", dv, "v"), ("dg", dg, "g"), ("dbeta", db, "beta")):
        out[name] = _together(s, w).view(s[like].shape)
    if s["start"] is not None:
        out["dh0"] = A
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("delta_fwd", "delta_train"):
        return _exact_delta(s, op == "delta_train")
    if op == "delta_step":
        pool = s["pool"].double()
        y = torch.zeros(s["v"].shape, dtype=torch.float64, device=pool.device)
        r = s["H"] // s["G"]
        for i, p in enumerate(s["at"].tolist()):
            if p >= 0:
                q, k = (s[w][i].double().repeat_interleave(r, 0) for w in ("q", "k"))
                pool[p], _ = _one_step(pool[p], k, s["v"][i].double(), torch.exp(s["g"][i].double()), s["beta"][i].double())
                y[i] = (pool[p] * q.unsqueeze(1)).sum(-1) / math.sqrt(s["K"])
        return {"y": y, "states": pool}
    a = s["x"].double()
    if s["r"] is not None:
        a = a + s["r"].double()
    w, size = s["weight"].double(), (a.square().sum(-1, keepdim=True) / case["cols"] + EPS).sqrt()
    unit = a / size
    y = unit * w
    if op == "norm_fwd":
        if case["out"] == "8bit":
            for c in range(0, case["cols"], BLOCK):
                top = y[:, c:c + BLOCK].abs().amax(-1, keepdim=True)
                step = (top / 127).clamp(min=1e-300)
                y[:, c:c + BLOCK] = torch.where(top < 2.0 ** -100, 0.0, torch.round(y[:, c:c + BLOCK] / step) * step)
        return {"y": y, "sum": a} if case["residual"] else {"y": y}
    d = s["dy"].double()
    out = {"y": y, "dweight": (d * unit).sum(0)}
    dunit = d * w
    out["dx"] = (dunit - unit * (dunit * unit).sum(-1, keepdim=True) / case["cols"]) / size
    if case["residual"]:
        out["dx"] += s["ds"].double()
        out["sum"] = a
    return out
