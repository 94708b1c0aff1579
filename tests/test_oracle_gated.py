"""The gated recurrence's oracle against closed forms and differences (CPU)."""
import numpy as np
import pytest

from oracle import gated


def _case(Bs=2, L=70, ED=3, seed=0, resets=False):
    r = np.random.default_rng(seed)
    inp = dict(x=r.standard_normal((Bs, L, ED)), gate_r=r.standard_normal((Bs, L, ED)),
               gate_i=r.standard_normal((Bs, L, ED)), lam=r.standard_normal(ED) - 3.0)
    reset = (r.random((Bs, L)) < 0.1).astype(np.uint8) if resets else None
    return inp, reset, r


def test_closed_form_of_constant_gates():
    """With constant gates and input h_t = a^t h0 + m s_i x (1 - a^t) / (1 - a)."""
    lam, c, gr, gi, x, h0 = 0.3, 2.0, -1.0, 0.5, 1.7, -0.4
    L = 40
    h = gated.gated_scan(np.full((1, L, 1), x), np.full((1, L, 1), gr), np.full((1, L, 1), gi),
                         np.array([lam]), c, h0=np.array([[h0]]))[0, :, 0]
    a = np.exp(-c * np.log1p(np.exp(lam)) / (1 + np.exp(-gr)))
    b = np.sqrt(1 - a * a) / (1 + np.exp(-gi)) * x
    t = np.arange(1, L + 1)
    assert np.allclose(h, a ** t * h0 + b * (1 - a ** t) / (1 - a), rtol=1e-12, atol=0)


def test_reset_starts_anew_whatever_was_before():
    inp, _, r = _case(L=20)
    reset = np.zeros((2, 20))
    reset[:, 7] = 1
    whole = gated.gated_scan(**inp, reset=reset, h0=np.full((2, 3), np.nan))
    assert np.isnan(whole[:, :7]).all()
    tail = {k: v[:, 7:] if v.ndim == 3 else v for k, v in inp.items()}
    first = reset[:, 7:]
    assert np.array_equal(whole[:, 7:], gated.gated_scan(**tail, reset=first))


@pytest.mark.parametrize("resets", [False, True])
def test_gradients_against_differences(resets):
    inp, reset, r = _case(resets=resets, seed=3)
    h0, w, wf = r.standard_normal((2, 3)), r.standard_normal((2, 70, 3)), r.standard_normal((2, 3))

    def loss(**kw):
        h0_ = kw.pop("h0", h0)
        h = gated.gated_scan(**{**inp, **kw}, reset=reset, h0=h0_)
        return (h * w).sum() + (h[:, -1] * wf).sum()

    h = gated.gated_scan(**inp, reset=reset, h0=h0)
    g = gated.gated_scan_bwd(**inp, dy=w, states=gated.kept_states(h, h0), reset=reset, dh_final=wf)
    eps = 1e-6
    for name, grad in (("x", "dx"), ("gate_r", "dgate_r"), ("gate_i", "dgate_i"), ("lam", "dlam"),
                       ("h0", "dh0")):
        base = h0 if name == "h0" else inp[name]
        for _ in range(6):
            d = r.standard_normal(base.shape)
            num = (loss(**{name: base + eps * d}) - loss(**{name: base - eps * d})) / (2 * eps)
            ana = (g[grad] * d).sum()
            # central differences: O(eps^2) truncation and 2^-52 |loss| / eps of rounding
            assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)) + 1e-8 * abs(loss()), (name, num, ana)


def test_ckpt8_rounds_to_half_a_step():
    x = np.random.default_rng(1).standard_normal((5, 130)).astype(np.float32)
    q, scale = gated.ckpt8(x)
    v = gated.ckpt8_values(q, scale)
    for k in range(3):
        part = slice(64 * k, 64 * (k + 1))
        # half a step, and the 32-bit rounding of the products
        assert (np.abs(v[:, part] - x[:, part]) <= 0.5001 * scale[k][:, None]).all()
        assert (np.abs(q[:, part]).max(1) == 127).all()
    q, scale = gated.ckpt8(np.zeros((2, 64), np.float32))
    assert not q.any() and not scale.any()


def test_pages():
    assert gated.pages_fork([1, 0, 1, 0], [2, 3, -1, 0]) == ([1, 1, 1, 1], [1, -1, 3, -1])
    assert gated.pages_compact([0, 1, 0, 0, 1, 1]) == ([1, 1, 1, 0, 0, 0], [-1, 1, -1, -1, 0, 2],
                                                       [(4, 0), (5, 2)])
