"""The gated delta rule where a block's system is at its worst: keys alike and beta
up to 2, so that writes are reflections and the inverse of the system has entries of
1 at every place.

Bound of the fp32 results of bf16 inputs (final states and their gradients): as in
test_gpu_delta.py, operands of 16 bits, 1e-5 of the 2-norm of the terms that are
summed.  The terms are not the result alone: with (I + A beta)^-1 = I - N beta and
W = V - Gam K S^T, a block sums S K^T (whose error goes through the inverse),
N (beta W) and (E beta X)^T K, and the adjoint likewise.  Reflections and decays
do not enlarge what earlier blocks are off by, so the blocks' squares add up.
fp32 inputs: sums of at most 64 terms in 2^-24 each are 64 2^-24 = 3.9e-6 of the same
terms, within the same bound.
"""
import numpy as np
import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from oracle import delta
from oracle.gated import f64
from test_gpu_delta import BF, F32, cuda, inputs

pytestmark = pytest.mark.gpu


def square(*terms):
    """The sum over all places of the product's terms' squares: `terms` as in a matrix product."""
    a, b = terms
    return ((a ** 2) @ (b ** 2))


def blocks(q, k, v, g, beta, dy, h0, dend, scale):
    """One head in 64 bits by blocks of 64 steps: (final state, bound's square, gradient of h0, bound's square)."""
    parts = []
    S, forward, back = h0, 0.0, 0.0
    for c in range(0, len(k), 64):
        at = slice(c, c + 64)
        K, Q, b, gam = k[at], q[at], beta[at, None], np.cumsum(g[at])
        D = np.tril(np.exp(np.minimum(gam[:, None] - gam[None], 0)))
        Gam, E = np.exp(gam)[:, None], np.exp(gam[-1] - gam)[:, None]
        A, P = np.tril(K @ K.T * D, -1), scale * np.tril(Q @ K.T * D)
        N = np.linalg.solve(np.eye(len(K)) + A * b.T, A)
        T = np.eye(len(K)) - N * b.T
        W = v[at] - Gam * (K @ S.T)
        X = T @ W
        dx = square(T, Gam * np.sqrt(square(K, S.T))) + square(N, b * W)
        forward += (square((E * b * X).T, K)).sum() + ((E * b) ** 2 * dx).sum()
        parts.append((K, Q, b, Gam, E, P, N, T))
        S = Gam[-1] * S + (E * b * X).T @ K
    end, A = S, dend
    for c, (K, Q, b, Gam, E, P, N, T) in reversed(list(enumerate(parts))):
        dY = dy[64 * c:64 * c + 64]
        dU = P.T @ dY + E * (K @ A.T)
        Z = T.T @ dU
        dz = square(T.T, np.sqrt(E ** 2 * square(K, A.T) + square(P.T, dY))) + square(N.T, b * dU)
        back += square((scale * Gam * dY).T, Q).sum() + square((Gam * b * Z).T, K).sum() + ((Gam * b) ** 2 * dz).sum()
        A = Gam[-1] * A + (scale * Gam * dY).T @ Q - (Gam * b * Z).T @ K
    return end, forward, A, back


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64), (40, 24)])
@pytest.mark.parametrize("beta,apart", [(2.0, 0.0), (1.9, 0.2), (1.0, 0.0), (2.0, None)])
@pytest.mark.parametrize("L", [64, 200])
def test_states(cuda_device, dtype, K, V, beta, apart, L):
    i, rest = inputs(1, 1, L, 2, 2, K, V, dtype)
    if apart is not None:
        k = 1.0 + apart * torch.randn(1, L, 2, K, generator=torch.Generator().manual_seed(2))
        i["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    i["beta"] = torch.full_like(i["beta"], beta)
    c = cuda(i, cuda_device)
    y, hf, saved = lrs.delta_rule_fwd(**c, scale=0.2, h0=rest["h0"].to(cuda_device), return_final_state=True, save="states")
    c.pop("v")
    dh0 = lrs.delta_rule_bwd(**c, dy=rest["dy"].to(cuda_device), saved=saved, scale=0.2,
                             dh_final=rest["dh_final"].to(cuda_device))["dh0"]
    exact = delta.delta_rule(**i, scale=0.2, h0=rest["h0"])["h_final"]
    for h in range(2):
        w = [f64(i[n])[0, :, h] for n in ("q", "k", "v", "g", "beta")]
        end, forward, first, back = blocks(*w, f64(rest["dy"])[0, :, h], f64(rest["h0"])[0, h], f64(rest["dh_final"])[0, h], 0.2)
        assert np.linalg.norm(end - exact[0, h]) <= 1e-10 * np.linalg.norm(end)       # the two 64-bit forms
        for got, want, terms in ((hf, end, forward), (dh0, first, back)):
            error = np.linalg.norm(got[0, h].double().cpu().numpy() - want)
            assert error <= 1e-5 * np.sqrt(terms + np.sum(want ** 2)), (error, np.sqrt(terms), np.linalg.norm(want))
