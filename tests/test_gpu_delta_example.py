"""The layer around the gated delta rule (GPU): norm, 8-bit input, delta rule
and norm together, trained on packed sequences and served from forked pages."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_rule.py")


def load():
    spec = importlib.util.spec_from_file_location("delta_rule_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(cuda_device):
    m = load()
    layer = m.Layer(48)
    losses = m.train(layer, 48, 4)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    # either way rounds h, its norm and the output to bf16, 2^-8 each at most; the norm's rows have a root mean square
    # of 1 and W_o keeps it, so the outputs stay below 8: three roundings of them, in either of the two
    assert m.serve(layer, 48) < 6 * 8 * 2.0 ** -8


def test_gradients_against_differences(cuda_device):
    """fp32 throughout but the 8-bit input, whose rounding the gradients take as none: so the differences are taken of
    the layer behind it, at the values that the 8 bits stand for, and of the norm on its own elsewhere."""
    m = load()
    layer = m.Layer(24, K=40, V=24, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(1, 150, 24, generator=g, device="cuda") for _ in range(2))
    offsets = torch.tensor([0, 67, 67, 150], dtype=torch.int32, device="cuda")
    dout, ds = (torch.randn(1, 150, 24, generator=g, device="cuda") for _ in range(2))
    out, s, _, kept = layer.forward(x, r, offsets, keep=True)
    grads = layer.backward(kept, dout, ds)
    u = m.lrs.ckpt8_load(*kept["u8"], torch.float32)

    def loss():
        heads, _ = layer._heads(u)
        y = m.lrs.delta_rule_fwd(*heads, offsets=offsets)
        n = m.lrs.rms_norm_fwd(y, layer.W["head_norm"])
        return ((n.flatten(-2) @ layer.W["o"]).double() * dout.double()).sum().item()

    for name in ("q", "k", "v", "g", "b", "o", "head_norm"):
        w, way = layer.W[name], torch.randn(layer.W[name].shape, generator=g, device="cuda")
        way = way / way.norm() * w.norm()
        e = 2e-3
        keep = w.clone()
        w.copy_(keep + e * way)
        up = loss()
        w.copy_(keep - e * way)
        down = loss()
        w.copy_(keep)
        want, got = (up - down) / (2 * e), (grads[name].double() * way.double()).sum().item()
        # the curve's third order, e^2, and the losses' own rounding, 2^-20 of their terms' sum over 2 e
        size = grads[name].norm().item() * way.norm().item()
        assert abs(got - want) <= 1e-3 * abs(want) + 2e-3 * size, (name, got, want, size)
    # the sum's own gradient goes straight through
    other = layer.backward(kept, dout, torch.zeros_like(ds))
    assert torch.allclose(grads["x"] - other["x"], ds, atol=1e-4)
