"""Refusals of the gated delta rule and of the norm (CPU only: no kernel is launched)."""
import ctypes

import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs

P = ctypes.c_void_p(0x10000)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3


def swapped(n, i, value):
    p = [P] * n
    p[i] = value
    return p


def fwd(ptrs=None, scale=1.0, Bs=1, L=8, G=2, H=4, K=16, V=8, n=1, bf16=1):
    p = ptrs or [P] * 12         # q k v g beta | offsets h0 y h_final states errors scratch
    return lrs.library().delta_rule_fwd(*p[:5], scale, *p[5:], Bs, L, G, H, K, V, n, bf16, None)


def bwd(ptrs=None, scale=1.0, Bs=1, L=8, G=2, H=4, K=16, V=8, n=1, bf16=1):
    p = ptrs or [P] * 16         # q k g beta | offsets dy dh_final states errors dq dk dv dg dbeta dh0 scratch
    return lrs.library().delta_rule_bwd(*p[:4], scale, *p[4:], Bs, L, G, H, K, V, n, bf16, None)


def step(ptrs=None, scale=1.0, Bs=2, G=2, H=4, K=16, V=8, pages=4, bf16=1):
    p = ptrs or [P] * 8          # q k v g beta | states pages y
    return lrs.library().delta_rule_step(*p[:5], scale, *p[5:], Bs, G, H, K, V, pages, bf16, None)


@pytest.mark.parametrize("call,n", [(fwd, 12), (bwd, 16)])
def test_sizes(call, n):
    for kw in (dict(L=0), dict(G=0), dict(H=0), dict(K=0), dict(V=-1), dict(Bs=2), dict(n=-1), dict(H=5), dict(G=3),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(L=2 ** 31, H=2 ** 40, G=2 ** 20)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=257), dict(V=257), dict(L=2 ** 31 - 1), dict(n=2 ** 31), dict(L=2 ** 30, H=2 ** 10)):
        assert call(**kw) == UNSUPPORTED, kw
    # offsets and the number of sequences go together
    assert call(n=0) == INVALID
    assert call(swapped(n, 5 if call is fwd else 4, None)) == INVALID


def test_fwd_pointers():
    for i in (0, 1, 2, 3, 4, 7, 9, 10, 11):      # states and errors: both or none
        assert fwd(swapped(12, i, None)) == INVALID
    for i in range(12):
        assert fwd(swapped(12, i, ODD)) == ALIGNMENT


def test_bwd_pointers():
    for i in (0, 1, 2, 3, 5, 7, 8, 9, 10, 11, 12, 13, 15):
        assert bwd(swapped(16, i, None)) == INVALID
    for i in range(16):
        assert bwd(swapped(16, i, ODD)) == ALIGNMENT
    assert bwd(swapped(16, 15, ctypes.c_void_p(0x10008))) == ALIGNMENT


def test_scratch_size():
    lib = lrs.library()
    for f in (lib.delta_rule_fwd_scratch, lib.delta_rule_bwd_scratch):
        assert f(1, 8, 2, 4, 16, 8, 0, 1) > 0 and f(1, 8, 2, 4, 17, 9, 3, 0) > 0
        assert f(1, 8, 3, 4, 16, 8, 0, 1) == f(1, 8, 2, 4, 300, 8, 0, 1) == 0
    assert lib.delta_rule_bwd_scratch(1, 8, 3, 4, 16, 8, 0, 1) == 0          # refused sizes
    assert lib.delta_rule_bwd_scratch(2, 8, 2, 4, 16, 8, 1, 1) == 0
    # a state a block of 64 steps and head at least
    assert lib.delta_rule_bwd_scratch(1, 2 ** 20, 8, 8, 128, 128, 0, 1) >= 2 ** 14 * 8 * 128 * 128 * 2


def test_step_refusals():
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert step(swapped(8, i, None)) == INVALID
    assert step(Bs=0) == step(pages=0) == step(H=5) == INVALID
    assert step(swapped(8, 6, None), pages=1) == INVALID       # fewer pages than rows
    assert step(pages=2 ** 24 + 1) == step(K=300) == UNSUPPORTED
    for i in range(8):
        assert step(swapped(8, i, ODD)) == ALIGNMENT


def norm(ptrs=None, eps=1e-6, rows=4, cols=8, bf16=1):
    p = ptrs or [P, P, P, P, P, None, None, P]      # x residual weight | sum y y_q y_scale rstd
    return lrs.library().rms_norm_fwd(*p[:3], eps, *p[3:], rows, cols, bf16, None)


def test_norm_refusals():
    usual = [P, P, P, P, P, None, None, P]
    for i, v in ((0, None), (1, None), (3, None), (4, None), (5, P), (6, P)):     # exactly one kind of output
        p = list(usual)
        p[i] = v
        assert norm(p) == INVALID, i
    for kw in (dict(rows=0), dict(cols=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(rows=2 ** 40, cols=2 ** 40)):
        assert norm(**kw) == INVALID, kw
    assert norm(rows=2 ** 31) == norm(cols=2 ** 31) == UNSUPPORTED
    for i in (0, 1, 2, 3, 4, 7):
        p = list(usual)
        p[i] = ODD
        assert norm(p) == ALIGNMENT, i
    f = lrs.library().rms_norm_bwd              # dy x residual weight rstd dsum dx dweight scratch
    for i in (0, 1, 4, 6, 8):
        assert f(*swapped(9, i, None), 4, 8, 1, None) == INVALID, i
    for i in range(9):
        assert f(*swapped(9, i, ODD), 4, 8, 1, None) == ALIGNMENT, i
    assert f(*[P] * 9, 0, 8, 1, None) == INVALID


@pytest.mark.parametrize("call", [
    lambda t: lrs.delta_rule_fwd(t(1, 4, 1, 8), t(1, 4, 1, 8), t(1, 4, 1, 8), t(1, 4, 1), t(1, 4, 1)),
    lambda t: lrs.delta_rule_bwd(t(1, 4, 1, 8), t(1, 4, 1, 8), t(1, 4, 1), t(1, 4, 1), t(1, 4, 1, 8), {}),
    lambda t: lrs.delta_rule_step(t(1, 1, 8), t(1, 1, 8), t(1, 1, 8), t(1, 1), t(1, 1), t(1, 1, 8, 8)),
    lambda t: lrs.rms_norm_fwd(t(4, 8)),
    lambda t: lrs.rms_norm_bwd(t(4, 8), t(4, 8), None, t(4)),
])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(torch.zeros)
