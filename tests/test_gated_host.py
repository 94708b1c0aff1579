"""Refusals of the gated recurrence, the 8-bit checkpoints and the state pages
(CPU only: no kernel is launched)."""
import ctypes

import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs

P = ctypes.c_void_p(0x10000)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
OK, INVALID, UNSUPPORTED, ALIGNMENT, NO_DEVICE = 0, 1, 2, 3, 6
END = OK if torch.cuda.is_available() else NO_DEVICE


def saved(**kw):
    o = lrs.GatedSaved()
    for k in ("states", "x_q", "r_q", "i_q", "x_s", "r_s", "i_s"):
        setattr(o, k, kw.get(k, 0x10000))
    return ctypes.byref(o)


def fwd(ptrs=None, c=8.0, keep=None, Bs=2, L=8, ED=4, bf16=1):
    p = ptrs or [P] * 8          # x gate_r gate_i lam reset h0 y h_final
    return lrs.library().gated_scan_fwd(*p[:4], c, *p[4:], keep, Bs, L, ED, bf16, None)


def bwd(ptrs=None, c=8.0, keep="all", Bs=2, L=8, ED=4, bf16=1):
    p = ptrs or [P] * 13         # x gate_r gate_i lam | reset dy dh_final | dx dr di dlam dh0 scratch
    keep = saved() if keep == "all" else keep
    return lrs.library().gated_scan_bwd(*p[:4], c, *p[4:7], keep, *p[7:], Bs, L, ED, bf16, None)


def step(ptrs=None, c=8.0, Bs=2, ED=4, pages=4, bf16=1):
    p = ptrs or [P] * 7          # x gate_r gate_i lam | states pages y
    return lrs.library().gated_scan_step(*p[:4], c, *p[4:], Bs, ED, pages, bf16, None)


def swapped(n, i, value):
    p = [P] * n
    p[i] = value
    return p


@pytest.mark.parametrize("c", [0.0, -1.0, float("nan"), float("inf")])
def test_constant_of_the_decay(c):
    assert fwd(c=c) == bwd(c=c) == step(c=c) == INVALID


def test_gated_fwd_refusals():
    for i in (0, 1, 2, 3, 6):
        assert fwd(swapped(8, i, None)) == INVALID
    for kw in (dict(Bs=0), dict(L=0), dict(ED=-1), dict(Bs=2 ** 15, L=2 ** 30, ED=2 ** 30)):
        assert fwd(**kw) == INVALID
    assert fwd(Bs=65536) == fwd(L=2 ** 31) == fwd(ED=2 ** 31) == UNSUPPORTED
    for i in (0, 1, 2, 3, 5, 6, 7):
        assert fwd(swapped(8, i, ODD)) == ALIGNMENT
    assert fwd(keep=saved(states=None)) == INVALID
    for k in ("x_q", "r_q", "i_q", "x_s", "r_s", "i_s"):     # all six or none
        assert fwd(keep=saved(**{k: None})) == INVALID
    assert fwd(keep=saved(states=0x10002)) == fwd(keep=saved(r_s=0x10002)) == ALIGNMENT


def test_gated_bwd_refusals():
    for i in (3, 5, 7, 8, 9, 10, 12):
        assert bwd(swapped(13, i, None)) == INVALID
    only = dict(x_q=None, r_q=None, i_q=None, x_s=None, r_s=None, i_s=None)
    for i in (0, 1, 2):          # read only without the 8-bit checkpoints
        assert bwd(swapped(13, i, None), keep=saved(**only)) == INVALID
    assert bwd(keep=None) == INVALID
    assert bwd(L=0) == INVALID and bwd(Bs=65536) == UNSUPPORTED
    for i in (3, 5, 6, 7, 8, 9, 10, 11, 12):
        assert bwd(swapped(13, i, ODD)) == ALIGNMENT


def test_step_refusals():
    for i in (0, 1, 2, 3, 4, 6):
        assert step(swapped(7, i, None)) == INVALID
    assert step(Bs=0) == step(pages=0) == INVALID
    assert step(swapped(7, 5, None), pages=1) == INVALID       # fewer pages than rows
    assert step(pages=2 ** 24 + 1) == UNSUPPORTED
    for i in (0, 3, 4, 5, 6):
        assert step(swapped(7, i, ODD)) == ALIGNMENT


def test_ckpt8_refusals():
    lib = lrs.library()
    for i in range(3):
        assert lib.ckpt8_save(*swapped(3, i, None), 4, 4, 1, None) == INVALID
        assert lib.ckpt8_load(*swapped(3, i, None), 4, 4, 1, None) == INVALID
    for f in (lib.ckpt8_save, lib.ckpt8_load):
        assert f(P, P, P, 0, 4, 1, None) == f(P, P, P, 4, 0, 1, None) == INVALID
        assert f(P, P, P, 2 ** 31, 4, 1, None) == f(P, P, P, 4, 2 ** 31, 1, None) == UNSUPPORTED
    assert lib.ckpt8_save(ODD, P, P, 4, 4, 1, None) == lib.ckpt8_save(P, P, ODD, 4, 4, 1, None) == ALIGNMENT
    assert lib.ckpt8_load(P, P, ODD, 4, 4, 1, None) == lib.ckpt8_load(P, ODD, P, 4, 4, 1, None) == ALIGNMENT


def test_pages_refusals():
    lib = lrs.library()
    sizes = (3, 1, 8, 64)        # n layers pages bytes
    for i in range(5):           # compact's last: scratch
        if i < 4:
            assert lib.state_pages_fork(*swapped(4, i, None), *sizes, None) == INVALID
        if i < 3:
            assert lib.state_pages_copy(*swapped(3, i, None), *sizes, None) == INVALID
        assert lib.state_pages_compact(*swapped(5, i, None), *sizes, None) == INVALID
    for bad in ((-1, 1, 8, 64), (3, 0, 8, 64), (3, 1, 0, 64), (3, 1, 8, 0), (3, 2 ** 40, 8, 2 ** 40)):
        assert lib.state_pages_fork(P, P, P, P, *bad, None) == INVALID
        assert lib.state_pages_copy(P, P, P, *bad, None) == INVALID
        assert lib.state_pages_compact(P, P, P, P, P, *bad, None) == INVALID
    assert lib.state_pages_fork(P, P, P, P, 3, 1, 2 ** 24 + 1, 4, None) == UNSUPPORTED
    assert lib.state_pages_fork(P, P, ODD, P, *sizes, None) == ALIGNMENT
    assert lib.state_pages_copy(P, P, ODD, *sizes, None) == ALIGNMENT
    assert lib.state_pages_compact(P, P, ODD, P, P, *sizes, None) == ALIGNMENT
    assert lib.state_pages_free(P, ODD, 3, 8, None) == ALIGNMENT
    assert lib.state_pages_free(None, P, 3, 8, None) == lib.state_pages_free(P, None, 3, 8, None) == INVALID
    # nothing to do: no list is needed
    assert lib.state_pages_free(P, None, 0, 8, None) == END
    assert lib.state_pages_fork(P, P, None, None, 0, 1, 8, 64, None) == END
    assert lib.state_pages_copy(P, None, None, 0, 1, 8, 64, None) == END


def test_valid_calls_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert fwd() == fwd(keep=saved()) == bwd() == step() == NO_DEVICE
    assert fwd(swapped(8, 4, None)) == NO_DEVICE
    assert lrs.library().ckpt8_save(P, P, P, 4, 4, 1, None) == NO_DEVICE
    assert lrs.library().state_pages_compact(P, P, P, None, P, 0, 1, 8, 64, None) == NO_DEVICE


T = torch.zeros


@pytest.mark.parametrize("call", [
    lambda: lrs.gated_scan_fwd(T(1, 2, 3), T(1, 2, 3), T(1, 2, 3), T(3)),
    lambda: lrs.gated_scan_bwd(T(1, 2, 3), T(1, 2, 3), T(1, 2, 3), T(3), T(1, 2, 3), {"states": T(1, 1, 3)}),
    lambda: lrs.gated_scan_step(T(2, 3), T(2, 3), T(2, 3), T(3), T(2, 3)),
    lambda: lrs.ckpt8_save(T(4, 4)),
    lambda: lrs.ckpt8_load(T(4, 4, dtype=torch.int8), T(1, 4)),
    lambda: lrs.state_pages_fork(T(4, 4), T(4, dtype=torch.uint8), T(1, dtype=torch.int32)),
    lambda: lrs.state_pages_copy(T(4, 4), T(1, dtype=torch.int32), T(1, dtype=torch.int32)),
    lambda: lrs.state_pages_free(T(4, dtype=torch.uint8), T(1, dtype=torch.int32)),
    lambda: lrs.state_pages_compact(T(4, 4), T(4, dtype=torch.uint8)),
])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensors"):
        call()


@pytest.mark.gpu
def test_python_refusals(cuda_device):
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=cuda_device)

    x, lam = t(2, 5, 8), t(8)
    good = dict(x=x, gate_r=x, gate_i=x, lam=lam)
    for bad, error in ((dict(gate_r=t(2, 5, 9)), ValueError), (dict(gate_i=t(2, 5, 8, dtype=torch.bfloat16)), TypeError),
                       (dict(lam=t(9)), ValueError), (dict(lam=t(8, dtype=torch.bfloat16)), TypeError),
                       (dict(x=t(5, 2, 8).transpose(0, 1)), ValueError), (dict(x=t(2, 5, 8, dtype=torch.float16)), TypeError),
                       (dict(reset=t(2, 4, dtype=torch.uint8)), ValueError), (dict(reset=t(2, 5)), TypeError),
                       (dict(h0=t(2, 9)), ValueError), (dict(save="4bit"), ValueError), (dict(y=t(2, 5, 9)), ValueError),
                       (dict(lam=None), TypeError), (dict(gate_r=None), TypeError), (dict(c=0.0), lrs.SsmError),
                       (dict(x=t(2, 0, 8), gate_r=t(2, 0, 8), gate_i=t(2, 0, 8)), lrs.SsmError)):
        with pytest.raises(error):
            lrs.gated_scan_fwd(**{**good, **bad})
    _, keep = lrs.gated_scan_fwd(**good, save="8bit")
    for bad, error in ((dict(dy=t(2, 5, 9)), ValueError), (dict(dy=t(2, 5, 8, dtype=torch.bfloat16)), ValueError),
                       (dict(saved={}), ValueError), (dict(saved=None), ValueError),
                       (dict(saved={"states": t(2, 2, 8)}), ValueError),
                       (dict(saved={k: v for k, v in keep.items() if k != "i_s"}), ValueError),
                       (dict(saved={**keep, "x_q": t(2, 5, 8)}), TypeError), (dict(dh_final=t(2, 7)), ValueError)):
        with pytest.raises(error):
            lrs.gated_scan_bwd(**{**good, "dy": x, "saved": {"states": keep["states"]}, **bad})
    row = dict(x=t(2, 8), gate_r=t(2, 8), gate_i=t(2, 8), lam=lam, states=t(4, 8))
    for bad, error in ((dict(states=t(4, 9)), ValueError), (dict(states=t(1, 8)), ValueError),
                       (dict(pages=t(3, dtype=torch.int32)), ValueError), (dict(pages=t(2, dtype=torch.int64)), TypeError)):
        with pytest.raises(error):
            lrs.gated_scan_step(**{**row, **bad})
    q, s = lrs.ckpt8_save(t(3, 70))
    for args, error in (((q, t(1, 3)), ValueError), ((q, s, torch.float16), TypeError), ((q.float(), s), TypeError)):
        with pytest.raises(error):
            lrs.ckpt8_load(*args)
    with pytest.raises(lrs.SsmError):
        lrs.ckpt8_save(t(0, 8))
    pool, used, pages = t(4, 6, 8), t(6, dtype=torch.uint8), t(2, dtype=torch.int32)
    for args, error in (((pool, t(4, dtype=torch.uint8), pages), ValueError), ((pool, used, pages.long()), TypeError),
                        ((pool.transpose(0, 1), used, pages), ValueError), ((pool, used, pages, 3), ValueError)):
        with pytest.raises(error):
            lrs.state_pages_fork(*args[:3], page_dim=args[3] if len(args) > 3 else 1)
    with pytest.raises(ValueError):
        lrs.state_pages_copy(pool, pages, t(3, dtype=torch.int32), page_dim=1)
