"""fp64 oracle of the gated linear recurrence, its 8-bit checkpoints and the
pages of a state cache: numpy, from the definitions, step by step.

  a_t = exp(-c softplus(lam) sigmoid(gate_r)),  m_t = sqrt(1 - a_t^2)
  h_t = a_t h_{t-1} + m_t sigmoid(gate_i) x_t       (reset: a_t = 0, m_t = 1)
"""
from __future__ import annotations

import numpy as np

BLOCK = 64


def f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu()
        a = a.double().numpy() if a.is_floating_point() else a.numpy()
    return np.asarray(a, dtype=np.float64)


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _softplus(v):
    return np.logaddexp(0.0, v)


def coefficients(gate_r, gate_i, lam, c, reset):
    """s_r, s_i, la, a, m; at a reset la = a = 0 and m = 1."""
    sr, si = _sigmoid(f64(gate_r)), _sigmoid(f64(gate_i))
    la = -c * _softplus(f64(lam)) * sr
    a, m = np.exp(la), np.sqrt(-np.expm1(2 * la))
    if reset is not None:
        cut = f64(reset)[..., None] != 0
        a, m, la = np.where(cut, 0.0, a), np.where(cut, 1.0, m), np.where(cut, 0.0, la)
    return sr, si, la, a, m


def gated_scan(x, gate_r, gate_i, lam, c=8.0, reset=None, h0=None):
    """Every state h (Bs, L, ED)."""
    x = f64(x)
    _, si, _, a, m = coefficients(gate_r, gate_i, lam, c, reset)
    cut = None if reset is None else f64(reset) != 0
    h = np.zeros_like(x)
    last = np.zeros_like(x[:, 0]) if h0 is None else f64(h0)
    for t in range(x.shape[1]):
        carried = a[:, t] * last
        if cut is not None:
            carried = np.where(cut[:, t, None], 0.0, carried)    # dropped, whatever it holds
        last = carried + m[:, t] * si[:, t] * x[:, t]
        h[:, t] = last
    return h


def kept_states(h, h0=None):
    """The states that enter the blocks of 64 steps."""
    first = np.zeros_like(h[:, 0]) if h0 is None else f64(h0)
    return np.stack([first] + [h[:, t - 1] for t in range(BLOCK, h.shape[1], BLOCK)], 1)


def gated_scan_bwd(x, gate_r, gate_i, lam, dy, states, c=8.0, reset=None, dh_final=None):
    """dict(dx, dgate_r, dgate_i, dlam, dh0), and ``size``: the sum of the
    absolute terms of dgate_r, elementwise, for error bounds."""
    x, dy, states, lam = f64(x), f64(dy), f64(states), f64(lam)
    sr, si, la, a, m = coefficients(gate_r, gate_i, lam, c, reset)
    cut = np.zeros(x.shape[:2], bool) if reset is None else f64(reset) != 0
    L = x.shape[1]
    before = np.zeros_like(x)
    for t in range(L):
        if t % BLOCK == 0:
            before[:, t] = states[:, t // BLOCK]
        else:
            carried = np.where(cut[:, t - 1, None], 0.0, a[:, t - 1] * before[:, t - 1])
            before[:, t] = carried + m[:, t - 1] * si[:, t - 1] * x[:, t - 1]
    g = np.zeros_like(x)
    u = np.zeros_like(x[:, 0]) if dh_final is None else f64(dh_final)
    for t in range(L - 1, -1, -1):
        g[:, t] = dy[:, t] + u
        u = np.where(cut[:, t, None], 0.0, a[:, t] * g[:, t])
    with np.errstate(divide="ignore", invalid="ignore"):
        # la / m -> 0 with la
        over = np.where(m > 0, la * a * a / m, 0.0)
        G = g * (la * a * before - over * si * x)
        size = np.abs(g) * (np.abs(la * a * before) + np.abs(over * si * x))
    G, size = np.where(cut[..., None], 0.0, G), np.where(cut[..., None], 0.0, size)
    sp = _softplus(lam)
    ratio = np.where(sp > 0, _sigmoid(lam) / np.where(sp > 0, sp, 1.0), 1.0)
    return dict(dx=g * m * si, dgate_r=G * (1 - sr), dgate_i=g * m * x * si * (1 - si),
                dlam=G.sum((0, 1)) * ratio, dh0=u, size=size, size_lam=size.sum((0, 1)) * ratio)


def ckpt8(x):
    """(q, scale) of the 8-bit checkpoint: 32-bit arithmetic, by its definition."""
    v = (x.detach().cpu().float().numpy() if hasattr(x, "detach") else np.asarray(x, np.float32))
    cols = v.shape[-1]
    v = v.reshape(-1, cols)
    groups = -(-cols // BLOCK)
    q, scale = np.zeros(v.shape, np.int8), np.zeros((groups, v.shape[0]), np.float32)
    one = np.float32
    for k in range(groups):
        part = v[:, k * BLOCK:(k + 1) * BLOCK]
        top = np.abs(part).max(1)
        small = top < one(2.0 ** -100)
        inv = np.where(small, one(0), one(127) / np.where(small, one(1), top)).astype(np.float32)
        scale[k] = np.where(small, one(0), top * one(1 / 127))
        q[:, k * BLOCK:(k + 1) * BLOCK] = np.rint(part * inv[:, None]).astype(np.int8)
    return q.reshape(x.shape), scale


def ckpt8_values(q, scale):
    """q * scale in 32 bits."""
    q = q.detach().cpu().numpy() if hasattr(q, "detach") else q
    scale = scale.detach().cpu().numpy() if hasattr(scale, "detach") else scale
    flat = q.reshape(-1, q.shape[-1])
    out = np.zeros(flat.shape, np.float32)
    for k in range(scale.shape[0]):
        part = slice(k * BLOCK, (k + 1) * BLOCK)
        out[:, part] = flat[:, part].astype(np.float32) * scale[k][:, None]
    return out.reshape(q.shape)


def pages_fork(used, src):
    """(used, dst) after a fork; used and src are lists."""
    start, used, dst = list(used), [int(bool(u)) for u in used], []
    for s in src:
        valid = s == -1 or (0 <= s < len(used) and start[s])
        page = used.index(0) if valid and 0 in used else -1
        if page >= 0:
            used[page] = 1
        dst.append(page)
    return used, dst


def pages_compact(used):
    """(used, moved, moves) after a compaction: moves is a list of (from, to)."""
    used = [int(bool(u)) for u in used]
    live = sum(used)
    holes = [p for p in range(live) if not used[p]]
    movers = [p for p in range(live, len(used)) if used[p]]
    moved = [p if used[p] else -1 for p in range(len(used))]
    for f, t in zip(movers, holes):
        moved[f] = t
    return [int(p < live) for p in range(len(used))], moved, list(zip(movers, holes))
