"""Pins of the gated delta rule's and the norm's oracle (CPU): special cases,
closed forms, a split of the sequence, and finite differences."""
import numpy as np
import pytest

from oracle import delta


def inputs(seed=0, Bs=2, L=9, G=2, H=4, K=5, V=3):
    r = np.random.default_rng(seed)
    k = r.normal(size=(Bs, L, G, K))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=r.normal(size=(Bs, L, G, K)), k=k, v=r.normal(size=(Bs, L, H, V)), g=-r.random((Bs, L, H)),
                beta=r.random((Bs, L, H)))


def test_a_unit_key_written_in_full_reads_back():
    i = inputs(1, Bs=1, L=1)
    i["beta"][:] = 1.0
    i["q"] = i["k"]
    S0 = np.random.default_rng(2).normal(size=(1, 4, 3, 5))
    assert np.allclose(delta.delta_rule(**i, scale=1.0, h0=S0)["y"], i["v"])     # whatever the state held


def test_orthogonal_keys_are_a_plain_sum():
    i = inputs(3, Bs=1, L=5, G=1, H=1)
    i["k"][0, :, 0] = np.eye(5)
    i["g"][:] = 0.0
    out = delta.delta_rule(**i)
    assert np.allclose(out["h_final"][0, 0], (i["beta"] * i["v"][..., 0, :])[0].T)


def test_no_write_is_decay_alone():
    i = inputs(4)
    i["beta"][:] = 0.0
    S0 = np.random.default_rng(5).normal(size=(2, 4, 3, 5))
    out = delta.delta_rule(**i, h0=S0)
    assert np.allclose(out["h_final"], S0 * np.exp(i["g"].sum(1))[..., None, None])


def test_split_and_packed_agree_with_the_whole():
    i = inputs(6, Bs=1, L=12)
    whole = delta.delta_rule(**i)
    first = delta.delta_rule(**{n: w[:, :7] for n, w in i.items()})
    rest = delta.delta_rule(**{n: w[:, 7:] for n, w in i.items()}, h0=first["h_final"])
    assert np.allclose(whole["y"][:, 7:], rest["y"]) and np.allclose(whole["h_final"], rest["h_final"])
    packed = delta.delta_rule(**i, offsets=np.array([1, 8, 8, 12]))
    alone = delta.delta_rule(**{n: w[:, 1:8] for n, w in i.items()})
    assert np.allclose(packed["y"][:, 1:8], alone["y"]) and np.all(packed["y"][:, :1] == 0)
    assert np.all(packed["h_final"][1] == 0)


def test_a_decay_of_zero_drops_the_state():
    i = inputs(7, Bs=1, L=6)
    i["g"][:, 3] = -np.inf
    S0 = np.full((1, 4, 3, 5), np.nan)
    out = delta.delta_rule(**i, h0=S0)
    alone = delta.delta_rule(**{n: w[:, 3:] for n, w in i.items()})
    assert np.allclose(out["y"][:, 3:], alone["y"])


def test_blocks_of_steps_agree_with_single_steps():
    """The block form that the kernels use."""
    i = inputs(8, Bs=1, L=20, G=1, H=1)
    q, k, v, g, b = (i[n][0, :, 0] for n in ("q", "k", "v", "g", "beta"))
    S0 = np.random.default_rng(9).normal(size=(1, 1, 3, 5))
    want = delta.delta_rule(**i, scale=1.0, h0=S0)
    gamma = np.cumsum(g)
    D = np.tril(np.exp(np.minimum(gamma[:, None] - gamma[None], 0)))
    Ab = np.tril(k @ k.T * D, -1)
    W = v - np.exp(gamma)[:, None] * (k @ S0[0, 0].T)
    X = np.linalg.solve(np.eye(20) + Ab * b, W)
    N = np.linalg.solve(np.eye(20) + Ab * b, Ab)
    assert np.allclose(X, W - N @ (b[:, None] * W)) and np.allclose(X, want["errors"][0, :, 0])
    U = b[:, None] * X
    assert np.allclose(np.exp(gamma)[:, None] * (q @ S0[0, 0].T) + (q @ k.T * D) @ U, want["y"][0, :, 0])
    S1 = np.exp(gamma[-1]) * S0[0, 0] + U.T @ (np.exp(gamma[-1] - gamma)[:, None] * k)
    assert np.allclose(S1, want["h_final"][0, 0])


@pytest.mark.parametrize("offsets", [None, np.array([1, 5, 5, 8])])
def test_gradients_against_differences(offsets):
    i = inputs(10, Bs=1 if offsets is not None else 2, L=9)
    r = np.random.default_rng(11)
    n = 3 if offsets is not None else 2
    i["h0"] = r.normal(size=(n, 4, 3, 5))
    dy, dend = r.normal(size=i["v"].shape), r.normal(size=i["h0"].shape)

    def loss(**w):
        o = delta.delta_rule(**w, offsets=offsets)
        return (o["y"] * dy).sum() + (o["h_final"] * dend).sum()

    got = delta.delta_rule_bwd(**i, dy=dy, offsets=offsets, dh_final=dend)
    for name, w in i.items():
        step = r.normal(size=w.shape)
        e = 1e-5
        diff = (loss(**dict(i, **{name: w + e * step})) - loss(**dict(i, **{name: w - e * step}))) / (2 * e)
        assert np.isclose((got["d" + name] * step).sum(), diff, rtol=1e-6, atol=1e-6), name


def test_norm_pins_and_gradients():
    r = np.random.default_rng(12)
    x, res, w = r.normal(size=(3, 7)), r.normal(size=(3, 7)), r.normal(size=7)
    y, s, rstd = delta.rms_norm(x, None, None, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0) and np.allclose(s, x)
    assert np.all(delta.rms_norm(np.zeros((2, 4)))[0] == 0)
    dy, ds = r.normal(size=(3, 7)), r.normal(size=(3, 7))

    def loss(x, w, res):
        y, s, _ = delta.rms_norm(x, w, res)
        return (y * dy).sum() + (s * ds).sum()

    dx, dw = delta.rms_norm_bwd(dy, x + res, w, ds)
    for name, at, grad in (("x", 0, dx), ("res", 2, dx), ("w", 1, dw)):
        args = [x, w, res]
        step, e = r.normal(size=args[at].shape), 1e-6
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + e * step, args[at] - e * step
        assert np.isclose((grad * step).sum(), (loss(*up) - loss(*down)) / (2 * e), rtol=1e-6, atol=1e-7), name
