"""A residual layer around the gated delta rule, trained and then served.

    s = x + residual;  u = norm(s);  q, k = unit rows of u W_q, u W_k
    h = delta rule(q, k, u W_v, g, beta);  out = norm of h's heads, times W_o

Training packs sequences of different lengths into one row and keeps the
layer's input u in 8 bits between its two passes; serving keeps one page of
state for each sequence and forks pages between tokens.  Run it on a GB300:

    python examples/delta_rule.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_ssm_gb300 as lrs  # noqa: E402


class Layer:
    """G key heads of K, H value heads of V on a stream of width d."""

    def __init__(self, d, G=2, H=4, K=64, V=64, seed=0, dtype=torch.bfloat16, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.sizes, self.dtype = (G, H, K, V), dtype
        wide = dict(q=G * K, k=G * K, v=H * V, g=H, b=H)
        self.W = {n: torch.randn(d, w, generator=g, device=device) / d ** 0.5 for n, w in wide.items()}
        self.W["o"] = torch.randn(H * V, d, generator=g, device=device) / (H * V) ** 0.5
        self.W["norm"] = torch.ones(d, device=device)
        self.W["head_norm"] = torch.ones(V, device=device)
        # rows of K columns become unit rows: their root mean square is 1 / sqrt(K)
        self.unit = torch.full((K,), K ** -0.5, device=device)

    def _heads(self, u):
        """q, k, v, g, beta of the layer's input u (..., d), and what their gradients need."""
        G, H, K, V = self.sizes
        u = u.float()
        raw = {n: (u @ self.W[n]).to(self.dtype) for n in "qkvgb"}
        lead = u.shape[:-1]
        rq, rk = raw["q"].view(*lead, G, K), raw["k"].view(*lead, G, K)
        q, sq = lrs.rms_norm_fwd(rq, self.unit, save=True)
        k, sk = lrs.rms_norm_fwd(rk, self.unit, save=True)
        gate = -torch.nn.functional.softplus(raw["g"].float() - 2.0)
        beta = torch.sigmoid(raw["b"].float())
        return (q, k, raw["v"].view(*lead, H, V), gate.to(self.dtype), beta.to(self.dtype)), (rq, sq, rk, sk, raw)

    def forward(self, x, residual, offsets=None, h0=None, keep=False):
        """(out, s, final states); with ``keep`` also what ``backward`` takes."""
        if keep:
            q8, s8, s, rstd = lrs.rms_norm_fwd(x, self.W["norm"], residual=residual, out="8bit", save=True)
            u = lrs.ckpt8_load(q8, s8, self.dtype)
        else:
            u, s = lrs.rms_norm_fwd(x, self.W["norm"], residual=residual)
        heads, more = self._heads(u)
        got = lrs.delta_rule_fwd(*heads, offsets=offsets, h0=h0, return_final_state=True,
                                 save="states" if keep else None)
        n, srow = lrs.rms_norm_fwd(got[0], self.W["head_norm"], save=True)
        out = (n.float().flatten(-2) @ self.W["o"]).to(self.dtype)
        if not keep:
            return out, s, got[1]
        q, k, _, gate, beta = heads
        return out, s, got[1], dict(x=x, residual=residual, rstd=rstd, u8=(q8, s8), q=q, k=k, gate=gate, beta=beta, more=more,
                                    y=got[0], n=n, srow=srow, saved=got[2], offsets=offsets)

    def backward(self, c, dout, ds):
        """Gradients of the weights by name, and "x" (the residual's too), for dout and ds, those of out and s."""
        G, H, K, V = self.sizes
        dout = dout.float()
        grads = {"o": c["n"].float().flatten(-2).flatten(0, -2).T @ dout.flatten(0, -2)}
        dn = (dout @ self.W["o"].T).to(self.dtype).view(c["n"].shape)
        norm = lrs.rms_norm_bwd(dn, c["y"], self.W["head_norm"], c["srow"])
        grads["head_norm"] = norm["dweight"]
        d = lrs.delta_rule_bwd(c["q"], c["k"], c["gate"], c["beta"], norm["dx"], c["saved"], offsets=c["offsets"],
                               need_dh0=False)
        rq, sq, rk, sk, raw = c["more"]
        draw = dict(v=d["dv"].flatten(-2).float())
        draw["q"] = lrs.rms_norm_bwd(d["dq"], rq, self.unit, sq, need_dweight=False)["dx"].flatten(-2).float()
        draw["k"] = lrs.rms_norm_bwd(d["dk"], rk, self.unit, sk, need_dweight=False)["dx"].flatten(-2).float()
        draw["g"] = -d["dg"].float() * torch.sigmoid(raw["g"].float() - 2.0)
        draw["b"] = d["dbeta"].float() * (b := torch.sigmoid(raw["b"].float())) * (1 - b)
        u = lrs.ckpt8_load(*c["u8"], self.dtype).float()
        flat = u.flatten(0, -2).T
        du = 0.0
        for n, w in draw.items():
            grads[n] = flat @ w.flatten(0, -2)
            du = du + w @ self.W[n].T
        first = lrs.rms_norm_bwd(du.to(self.dtype), c["x"], self.W["norm"], c["rstd"], residual=c["residual"], ds=ds)
        grads["norm"], grads["x"] = first["dweight"], first["dx"]
        return grads

    def step(self, x, residual, states, pages):
        """(out, s) of one token a row; the states move on in their pages."""
        u, s = lrs.rms_norm_fwd(x, self.W["norm"], residual=residual)
        heads, _ = self._heads(u)
        y = lrs.delta_rule_step(*heads, states, pages)
        return (lrs.rms_norm_fwd(y, self.W["head_norm"]).float().flatten(-2) @ self.W["o"]).to(self.dtype), s


def train(layer, d, steps, lengths=(70, 129, 1, 200), lr=3e-3, seed=1):
    """Losses of recalling each channel's value three tokens back, by gradient descent with momentum."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ends = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    total, speed, losses = int(sum(lengths)), {n: torch.zeros_like(w) for n, w in layer.W.items()}, []
    for _ in range(steps):
        x = torch.randn(1, total, d, generator=g, device="cuda").to(layer.dtype)
        target = torch.roll(x.float(), 3, 1)
        out, _, _, kept = layer.forward(x, torch.zeros_like(x), ends, keep=True)
        diff = out.float() - target
        grads = layer.backward(kept, 2.0 / diff.numel() * diff, None)
        for n, w in layer.W.items():
            speed[n].mul_(0.9).add_(grads[n])
            w -= lr * diff.shape[1] ** 0.5 * speed[n]
        losses.append(diff.square().mean())
    return torch.stack(losses).tolist()


def serve(layer, d, requests=3, prompt=75, tokens=5, num_pages=16, seed=2):
    """Prompts, each continued twice from forked pages; the largest difference
    between the steps' outputs and those of whole passes over the same tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, H, K, V = layer.sizes
    x = torch.randn(requests, prompt, d, generator=g, device="cuda").to(layer.dtype)
    pool = torch.zeros(num_pages, H, V, K, device="cuda")
    used = torch.zeros(num_pages, dtype=torch.uint8, device="cuda")
    _, _, state = layer.forward(x, torch.zeros_like(x))
    first = lrs.state_pages_fork(pool, used, torch.full((requests,), -1, dtype=torch.int32, device="cuda"))
    pool[first.long()] = state
    pages = torch.cat((first, lrs.state_pages_fork(pool, used, first)))
    more = torch.randn(2 * requests, tokens, d, generator=g, device="cuda").to(layer.dtype)
    got = torch.stack([layer.step(more[:, t].contiguous(), torch.zeros_like(more[:, t]), pool, pages)[0]
                       for t in range(tokens)], 1)
    whole = torch.cat((torch.cat((x, x)), more), 1)
    want, _, _ = layer.forward(whole, torch.zeros_like(whole))
    return (got.float() - want[:, prompt:].float()).abs().max().item()


def main():
    d = 64
    layer = Layer(d)
    losses = train(layer, d, 60)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    print("largest difference between steps and whole passes: %.2e" % serve(layer, d))
    lrs.ssm_check_device_errors()


if __name__ == "__main__":
    main()
