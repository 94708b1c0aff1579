"""fp64 oracle of the gated delta rule and of the root-mean-square norm:
numpy, from the definitions, step by step.

  x_t = v_t - a_t S_{t-1} k_t,  S_t = a_t S_{t-1} + beta_t x_t k_t^T,  y_t = scale S_t q_t,  a_t = e^(g_t)
"""
from __future__ import annotations

import numpy as np

from oracle.gated import f64

BLOCK = 64


def spans(q_shape, offsets):
    """[(row of the batch, first token, end)] of every sequence."""
    if offsets is None:
        return [(b, 0, q_shape[1]) for b in range(q_shape[0])]
    o = [int(v) for v in np.asarray(offsets.cpu() if hasattr(offsets, "cpu") else offsets)]
    return [(0, a, b) for a, b in zip(o, o[1:])]


def _heads(w, H):
    """(L, G, K) -> (H, L, K), each head with its group's rows."""
    return np.repeat(w, H // w.shape[1], axis=1).transpose(1, 0, 2)


def _walk(q, k, v, g, beta, S, scale):
    """One sequence: q, k (H, L, K), v (H, L, V), g, beta (H, L).  y, x and every state, the one before included."""
    with np.errstate(over="ignore"):
        a = np.exp(g)
    H, L, _ = q.shape
    y, x, states = np.zeros_like(v), np.zeros_like(v), np.zeros((L + 1,) + S.shape)
    states[0] = S
    for t in range(L):
        S = np.where((a[:, t] == 0)[:, None, None], 0.0, S) * a[:, t, None, None]    # dropped, whatever it holds
        x[:, t] = v[:, t] - np.einsum("hvk,hk->hv", S, k[:, t])
        S = S + np.einsum("hv,hk->hvk", beta[:, t, None] * x[:, t], k[:, t])
        y[:, t] = scale * np.einsum("hvk,hk->hv", S, q[:, t])
        states[t + 1] = S
    return y, x, states


def rounded(k, g, beta, x, states):
    """Where the state before a block of 64 steps, and the writes u inside it, are rounded on their own, S is off by the
    sum of those errors, whatever is left of S: the squares of the terms, (L + 1, H, V, K)."""
    a2, u2 = np.exp(2 * g), (beta[..., None] * x) ** 2
    E = np.zeros_like(states)
    for t in range(states.shape[0]):
        if t % BLOCK == 0:
            E[t] = states[t] ** 2
        else:
            E[t] = a2[:, t - 1, None, None] * E[t - 1] + np.einsum("hv,hk->hvk", u2[:, t - 1], k[:, t - 1] ** 2)
    return E


def delta_rule(q, k, v, g, beta, scale=None, offsets=None, h0=None):
    """dict(y, h_final, errors, states) with the states before steps 0, 64, ... of every sequence in a list, and
    y_terms, the 2-norms of the terms whose sums y are (see ``rounded``)."""
    q, k, v, g, beta, h0 = (f64(w) for w in (q, k, v, g, beta, h0))
    H, V, K = v.shape[2], v.shape[3], q.shape[3]
    scale = K ** -0.5 if scale is None else scale
    seqs = spans(q.shape, offsets)
    out = dict(y=np.zeros_like(v), y_terms=np.zeros_like(v), errors=np.zeros_like(v), h_final=np.zeros((len(seqs), H, V, K)), states=[])
    for i, (b, first, end) in enumerate(seqs):
        S = np.zeros((H, V, K)) if h0 is None else h0[i]
        at = (b, slice(first, end))
        y, x, states = _walk(_heads(q[at], H), _heads(k[at], H), v[at].transpose(1, 0, 2), g[at].T, beta[at].T, S, scale)
        out["y"][at], out["errors"][at] = y.transpose(1, 0, 2), x.transpose(1, 0, 2)
        E = rounded(_heads(k[at], H), g[at].T, beta[at].T, x, states)
        # after step t: the block's first state and its writes up to t
        last = np.exp(2 * g[at].T).transpose(1, 0)[..., None, None] * E[:-1] + np.einsum(
            "htv,htk->thvk", (beta[at].T[..., None] * x) ** 2, _heads(k[at], H) ** 2)
        out["y_terms"][at] = scale * np.sqrt(np.einsum("thvk,htk->thv", last, _heads(q[at], H) ** 2))
        out["h_final"][i] = states[-1]
        out["states"].append(states[:-1:BLOCK])
    return out


def delta_rule_bwd(q, k, v, g, beta, dy, scale=None, offsets=None, h0=None, dh_final=None):
    """dict(dq, dk, dv, dg, dbeta, dh0), and dq_terms, dk_terms, dg_terms, dbeta_terms: the 2-norms of the terms whose
    signed sums those are, which the sums may fall far below (see ``rounded``)."""
    q, k, v, g, beta, dy, h0, dh_final = (f64(w) for w in (q, k, v, g, beta, dy, h0, dh_final))
    H, V, G, K = v.shape[2], v.shape[3], q.shape[2], q.shape[3]
    scale = K ** -0.5 if scale is None else scale
    seqs = spans(q.shape, offsets)
    out = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dg=np.zeros_like(g),
               dbeta=np.zeros_like(beta), dq_terms=np.zeros_like(q), dk_terms=np.zeros_like(k),
               dg_terms=np.zeros_like(g), dbeta_terms=np.zeros_like(beta), dh0=np.zeros((len(seqs), H, V, K)))
    for i, (b, first, end) in enumerate(seqs):
        at = (b, slice(first, end))
        qs, ks, vs, ds = _heads(q[at], H), _heads(k[at], H), v[at].transpose(1, 0, 2), dy[at].transpose(1, 0, 2)
        gs, bs = g[at].T, beta[at].T
        S = np.zeros((H, V, K)) if h0 is None else h0[i]
        _, x, states = _walk(qs, ks, vs, gs, bs, S, scale)
        A = np.zeros((H, V, K)) if dh_final is None else dh_final[i].copy()
        E = rounded(ks, gs, bs, x, states)
        F = A * A                   # the same for A: the adjoint behind the block, and what the block subtracts
        for t in range(end - first - 1, -1, -1):
            a = np.exp(gs[:, t])[:, None, None]
            old = np.where(a == 0, 0.0, states[t]) * a
            dq = scale * np.einsum("hvk,hv->hk", states[t + 1], ds[:, t])
            A = A + scale * np.einsum("hv,hk->hvk", ds[:, t], qs[:, t])
            du = np.einsum("hvk,hk->hv", A, ks[:, t])
            u, dx = bs[:, t, None] * x[:, t], bs[:, t, None] * du
            dk = np.einsum("hvk,hv->hk", A, u) - np.einsum("hvk,hv->hk", old, dx)
            row, before = (b, first + t), E[t] * a * a
            if t % BLOCK == BLOCK - 1:
                F = A * A
            sums = lambda f, w: np.einsum(f, w[0] ** 2, w[1])  # noqa: E731
            out["dq_terms"][row] += scale * np.sqrt(sums("hv,hvk->hk", (ds[:, t], before + np.einsum("hv,hk->hvk", u ** 2, ks[:, t] ** 2)))).reshape(G, -1, K).sum(1)
            dk2 = sums("hv,hvk->hk", (u, F)) + sums("hv,hvk->hk", (dx, before))
            out["dk_terms"][row] += np.sqrt(dk2).reshape(G, -1, K).sum(1)
            out["dbeta_terms"][row] = np.sqrt((x[:, t] ** 2 * (sums("hk,hvk->hv", (ks[:, t], F)) + du ** 2)).sum(-1))
            A = A - np.einsum("hv,hk->hvk", dx, ks[:, t])
            F = F + np.einsum("hv,hk->hvk", dx ** 2, ks[:, t] ** 2)
            out["dq"][row] += dq.reshape(G, -1, K).sum(1)
            out["dk"][row] += dk.reshape(G, -1, K).sum(1)
            out["dv"][row], out["dbeta"][row] = dx, (du * x[:, t]).sum(-1)
            out["dg"][row] = (A * old).sum((-2, -1))
            out["dg_terms"][row] = np.sqrt((np.abs(A * old).sum(-1) ** 2).sum(-1) +
                                           (A ** 2 * before + F * old ** 2).sum((-2, -1)))
            A, F = A * a, F * a ** 2
        out["dh0"][i] = A
    return out


def delta_rule_step(q, k, v, g, beta, states, pages, scale=None):
    """(y, states) after one token."""
    q, k, v, g, beta, states = (f64(w) for w in (q, k, v, g, beta, states))
    states, y = states.copy(), np.zeros_like(v)
    pages = range(q.shape[0]) if pages is None else [int(p) for p in pages]
    for b, p in enumerate(pages):
        if 0 <= p < states.shape[0]:
            one = delta_rule(q[b][None, None], k[b][None, None], v[b][None, None], g[b][None, None], beta[b][None, None],
                             scale, None, states[p][None])
            y[b], states[p] = one["y"][0, 0], one["h_final"][0]
    return y, states


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, s, r)."""
    s = f64(x) + (0.0 if residual is None else f64(residual))
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s * r * (1.0 if weight is None else f64(weight)), s, r[..., 0]


def rms_norm_bwd(dy, s, weight=None, ds=None, eps=1e-6):
    """(dx, dweight)."""
    s, dy = f64(s), f64(dy)
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    wd = dy * (1.0 if weight is None else f64(weight))
    dx = r * (wd - s * r * r * (wd * s).mean(-1, keepdims=True)) + (0.0 if ds is None else f64(ds))
    return dx, (dy * s * r).reshape(-1, s.shape[-1]).sum(0)
