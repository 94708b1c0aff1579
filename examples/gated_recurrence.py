"""A layer around the gated linear recurrence, trained and then served.

Training keeps what the backward pass needs in 8 bits; serving keeps one page
of state for each sequence and forks, frees and compacts the pages between
tokens.  Run it on a GB300:

    python examples/gated_recurrence.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_ssm_gb300 as lrs  # noqa: E402


class Layer:
    """out = h W_out with h the gated recurrence over x W_in, gated by x W_r and x W_i."""

    def __init__(self, d, width, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.W = {k: torch.randn(d, width, generator=g, device=device) / d ** 0.5 for k in ("in", "r", "i")}
        self.W["out"] = torch.randn(width, d, generator=g, device=device) / width ** 0.5
        # decays between 0.9 and 0.999 where the gate is open
        a = 0.9 + 0.099 * torch.rand(width, generator=g, device=device)
        self.W["lam"] = torch.log(torch.expm1(-torch.log(a) / 8.0))
        self.moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.W.items()}
        self.t = 0

    def inputs(self, x):
        """x W_in, x W_r and x W_i in bf16; x is (..., d)."""
        return [(x @ self.W[k]).to(torch.bfloat16) for k in ("in", "r", "i")]

    def train_step(self, x, target, lr=1e-2):
        """One step of Adam on the mean squared error; returns the loss (a tensor)."""
        u, r, i = self.inputs(x)
        h, saved = lrs.gated_scan_fwd(u, r, i, self.W["lam"], save="8bit")
        del u, r, i                      # the checkpoint stands for them
        h32 = h.float()
        diff = h32 @ self.W["out"] - target
        dout = 2.0 / diff.numel() * diff
        dh = (dout @ self.W["out"].T).to(torch.bfloat16)
        g = lrs.gated_scan_bwd(None, None, None, self.W["lam"], dh, saved)
        flat = x.reshape(-1, x.shape[-1]).T
        grads = {k: flat @ g[n].float().reshape(-1, g[n].shape[-1])
                 for k, n in (("in", "dx"), ("r", "dgate_r"), ("i", "dgate_i"))}
        grads["out"] = h32.reshape(-1, h.shape[-1]).T @ dout.reshape(-1, dout.shape[-1])
        grads["lam"] = g["dlam"]
        self.t += 1
        for k, w in self.W.items():
            m, v = self.moments[k]
            m.lerp_(grads[k], 0.1)
            v.lerp_(grads[k] ** 2, 0.01)
            w -= lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8)
        return diff.square().mean()

    def prefill(self, x):
        """Outputs (Bs, L, d) and final states (Bs, width) of whole prompts."""
        h, state = lrs.gated_scan_fwd(*self.inputs(x), self.W["lam"], return_final_state=True)
        return h.float() @ self.W["out"], state

    def step(self, x, states, pages):
        """Outputs (Bs, d) of one token a row; the states move on in their pages."""
        h = lrs.gated_scan_step(*self.inputs(x), self.W["lam"], states, pages)
        return h.float() @ self.W["out"]


def averages(x, decay):
    """The target: running averages of x's channels, y_t = decay y_{t-1} + (1 - decay) x_t."""
    y, last = torch.empty_like(x), torch.zeros_like(x[:, 0])
    for t in range(x.shape[1]):
        last = decay * last + (1 - decay) * x[:, t]
        y[:, t] = last
    return y


def train(layer, d, steps, Bs=8, L=200, seed=1):
    """The losses of `steps` steps on fresh random sequences."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for _ in range(steps):
        x = torch.randn(Bs, L, d, generator=g, device="cuda")
        losses.append(layer.train_step(x, averages(x, 0.95)))
    return torch.stack(losses).tolist()


def serve(layer, d, requests=5, prompt=37, tokens=6, num_pages=32, seed=2):
    """Prompts, each continued twice; the second continuations end half-way and
    the pool is made dense again.  Returns the largest difference between the
    outputs of the steps and those of whole scans over the same tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(requests, prompt, d, generator=g, device="cuda")
    pool = torch.zeros(num_pages, layer.W["lam"].shape[0], device="cuda")
    used = torch.zeros(num_pages, dtype=torch.uint8, device="cuda")
    _, state = layer.prefill(x)
    first = lrs.state_pages_fork(pool, used, torch.full((requests,), -1, dtype=torch.int32, device="cuda"))
    pool[first.long()] = state
    second = lrs.state_pages_fork(pool, used, first)          # the same prompts, continued otherwise
    pages = torch.cat((first, second))
    more = torch.randn(2 * requests, tokens, d, generator=g, device="cuda")
    got = torch.empty(2 * requests, tokens, d, device="cuda")
    half = tokens // 2
    for t in range(half):
        got[:, t] = layer.step(more[:, t].contiguous(), pool, pages)
    lrs.state_pages_free(used, first)                         # the first continuations end
    live = second.clone()
    lrs.state_pages_compact(pool, used, live)
    for t in range(half, tokens):
        got[requests:, t] = layer.step(more[requests:, t].contiguous(), pool, live)
    want, _ = layer.prefill(torch.cat((torch.cat((x, x)), more), 1))
    want = want[:, prompt:]
    return max((got[:, :half] - want[:, :half]).abs().max().item(),
               (got[requests:, half:] - want[requests:, half:]).abs().max().item())


def main():
    d = 16
    layer = Layer(d, 256)
    losses = train(layer, d, 150)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    print("largest difference between steps and whole scans: %.2e" % serve(layer, d))
    lrs.ssm_check_device_errors()


if __name__ == "__main__":
    main()
