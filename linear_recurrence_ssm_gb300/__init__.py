"""GB300-native selective-scan linear recurrence: a thin Python binding of
libssmscan.so (C ABI declared in include/ssm_scan.h).

Every call marshals torch CUDA tensors into raw device pointers plus the
current CUDA stream and calls the C entry point of the same name; all of the
computation runs in the library's sm_103a kernels.  There is no fallback: if
the library is missing or fails to load, importing a function raises.

Functions
---------
ssm_scan_fwd(x, delta, A, B, C, D=None, y=None, **options)
    Diagonal-A selective scan (shape API of selective_scan in "scan output is
    different between sequential and parallel versions", mamba.py issue 26).
    x, delta: (Bs, L, ED); A: (ED, N) fp32; B, C: (Bs, L, N); D: (ED) fp32.
    fp32 inputs call the C ``ssm_scan_fwd``; bf16 inputs call
    ``ssm_scan_fwd_bf16``.  Returns y (Bs, L, ED) fp32.
ssd_chunk_scan_fwd(x, dt, A_head, B, C, D=None, chunk=256, bidirectional=False, y=None, **options)
    Chunked scalar-decay scan ("Some questions of Bi-Mamba2 and Hydra",
    Bi-Mamba2 issue 1).  x: (Bs, L, H, P) bf16 or fp32; dt: (Bs, L, H), same type;
    A_head: (H) fp32; B, C: (Bs, L, N) or (Bs, L, G, N) bf16 (head h reads
    group h // (H // G)); D: (H) fp32.  Returns y (Bs, L, H, P) fp32.

gated_scan_fwd(x, gate_r, gate_i, lam, c=8.0, ...), gated_scan_bwd, gated_scan_step
    Gated linear recurrence (one decay per channel and step, set by a gate):
    forward, gradients, and one token for rows whose states lie in pages.
ckpt8_save(x), ckpt8_load(q, scale, dtype)
    8-bit activation checkpoints; ``gated_scan_fwd(..., save="8bit")`` keeps
    its inputs this way and ``gated_scan_bwd`` reads them so.
state_pages_fork / _copy / _free / _compact
    The pages of a state cache.

Options (of the selective scans; any of them selects the ``*_ex`` C entry point):
``dt_bias`` (ED or H, fp32), ``dt_softplus``, ``dt_limit=(lo, hi)``, ``z``
(shaped and typed like x), ``h0`` (fp32 initial state, (Bs, ED, N) or
(Bs, H, P, N)) and ``return_final_state`` (the call then returns
``(y, h_final)``).
"""
from __future__ import annotations

import ctypes
import math
import os

from . import _build

__all__ = ["ssm_scan_fwd", "ssm_scan_fwd_bf16", "ssd_chunk_scan_fwd", "ssm_check_device_errors",
           "ssm_scan_fwd_plan", "ssm_scan_bwd", "ssd_chunk_scan_bwd", "ScanOptions",
           "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "GatedSaved", "ckpt8_save",
           "ckpt8_load", "state_pages_fork", "state_pages_copy", "state_pages_free",
           "state_pages_compact",
           "SsmError", "library", "build", "status_string", "STATUS"]

STATUS = {
    0: "SSM_OK", 1: "SSM_ERR_INVALID_ARG", 2: "SSM_ERR_UNSUPPORTED", 3: "SSM_ERR_ALIGNMENT",
    4: "SSM_ERR_CUDA", 5: "SSM_ERR_DEVICE_TIMEOUT", 6: "SSM_ERR_NO_DEVICE",
}

# Every symbol include/ssm_scan.h declares, with its ctypes signature.
_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
SIGNATURES = {
    "ssm_scan_fwd": ([_VP] * 7 + [_I64] * 4 + [_VP], ctypes.c_int),
    "ssm_scan_fwd_bf16": ([_VP] * 7 + [_I64] * 4 + [_VP], ctypes.c_int),
    "ssd_chunk_scan_fwd": ([_VP] * 7 + [_I64] * 6 + [ctypes.c_int, _VP], ctypes.c_int),
    "ssd_chunk_scan_fwd_noalloc": ([_VP] * 7 + [_I64] * 6 + [ctypes.c_int, _VP], ctypes.c_int),
    "ssm_scan_fwd_plan": ([_I64] * 4 + [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int32)] * 3,
                          ctypes.c_int),
    "ssm_scan_fwd_ex": ([_VP] * 7 + [_I64] * 4 + [ctypes.c_int, _VP, _VP], ctypes.c_int),
    "ssm_scan_bwd": ([_VP] * 13 + [_I64] * 4 + [ctypes.c_int, _VP], ctypes.c_int),
    "ssd_chunk_scan_bwd": ([_VP] * 13 + [_I64] * 6 + [ctypes.c_int, ctypes.c_int, _VP], ctypes.c_int),
    "ssm_scan_bwd_ex": ([_VP] * 16 + [_I64] * 4 + [ctypes.c_int, _VP, _VP], ctypes.c_int),
    "ssd_chunk_scan_bwd_ex": ([_VP] * 16 + [_I64] * 5 + [ctypes.c_int, ctypes.c_int, _VP, _VP],
                              ctypes.c_int),
    "ssd_chunk_scan_fwd_ex": ([_VP] * 7 + [_I64] * 6 + [ctypes.c_int, ctypes.c_int, _VP, _VP],
                              ctypes.c_int),
    "gated_scan_fwd": ([_VP] * 4 + [_F32] + [_VP] * 5 + [_I64] * 3 + [ctypes.c_int, _VP], ctypes.c_int),
    "gated_scan_bwd": ([_VP] * 4 + [_F32] + [_VP] * 10 + [_I64] * 3 + [ctypes.c_int, _VP], ctypes.c_int),
    "gated_scan_step": ([_VP] * 4 + [_F32] + [_VP] * 3 + [_I64] * 3 + [ctypes.c_int, _VP], ctypes.c_int),
    "ckpt8_save": ([_VP] * 3 + [_I64] * 2 + [ctypes.c_int, _VP], ctypes.c_int),
    "ckpt8_load": ([_VP] * 3 + [_I64] * 2 + [ctypes.c_int, _VP], ctypes.c_int),
    "state_pages_fork": ([_VP] * 4 + [_I64] * 4 + [_VP], ctypes.c_int),
    "state_pages_copy": ([_VP] * 3 + [_I64] * 4 + [_VP], ctypes.c_int),
    "state_pages_free": ([_VP] * 2 + [_I64] * 2 + [_VP], ctypes.c_int),
    "state_pages_compact": ([_VP] * 5 + [_I64] * 4 + [_VP], ctypes.c_int),
    "ssm_check_device_errors": ([_VP], ctypes.c_int),
    "ssm_selftest_wait_timeout": ([_VP], ctypes.c_int),
    "gated_selftest_wait_timeout": ([ctypes.c_int, ctypes.c_int, _VP], ctypes.c_int),
    "ssm_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "ssm_version": ([], ctypes.c_int),
}

_lib = None


class ScanOptions(ctypes.Structure):
    """ssm_scan_options_t of include/ssm_scan.h."""
    _fields_ = [("dt_bias", _VP), ("dt_softplus", ctypes.c_int32), ("dt_limit", ctypes.c_int32),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float), ("z", _VP),
                ("h0", _VP), ("h_final", _VP), ("ngroups", ctypes.c_int32)]


_OPTION_KEYS = ("dt_bias", "dt_softplus", "dt_limit", "z", "h0", "return_final_state")


def _options(x, channels, state_shape, dev, dt_bias=None, dt_softplus=False, dt_limit=None,
             z=None, h0=None, return_final_state=False, ngroups=1):
    """Validate the options and build (ScanOptions, h_final tensor or None, keep-alive list)."""
    import torch
    o = ScanOptions()
    keep = []
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", (torch.float32,), dev, (1,))
        if dt_bias.shape[0] != channels:
            raise ValueError("dt_bias must have %d entries" % channels)
        o.dt_bias = dt_bias.data_ptr()
        keep.append(dt_bias)
    o.dt_softplus = 1 if dt_softplus else 0
    if dt_limit is not None:
        o.dt_limit = 1
        o.dt_min, o.dt_max = float(dt_limit[0]), float(dt_limit[1])
    if z is not None:
        _check(z, "z", (x.dtype,), dev)
        if z.shape != x.shape:
            raise ValueError("z must have the shape of x")
        o.z = z.data_ptr()
        keep.append(z)
    if h0 is not None:
        _check(h0, "h0", (torch.float32,), dev)
        if tuple(h0.shape) != tuple(state_shape):
            raise ValueError("h0 must have shape %s" % (tuple(state_shape),))
        o.h0 = h0.data_ptr()
        keep.append(h0)
    o.ngroups = int(ngroups)
    hf = None
    if return_final_state:
        hf = torch.empty(state_shape, dtype=torch.float32, device=dev)
        o.h_final = hf.data_ptr()
    return o, hf, keep


class GatedSaved(ctypes.Structure):
    """gated_scan_saved_t of include/ssm_scan.h."""
    _fields_ = [(n, _VP) for n in ("states", "x_q", "r_q", "i_q", "x_s", "r_s", "i_s")]


class SsmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s" % (fn, status_string(status)))


def build(force: bool = False) -> str:
    """Compile libssmscan.so in-tree (nvcc, sm_103a)."""
    return _build.build(force=force)


def library() -> ctypes.CDLL:
    """The loaded C library (built first if its sources are newer)."""
    global _lib
    if _lib is None:
        path = _build.LIB_PATH
        if _build.needs_build():
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError("libssmscan.so is missing and could not be built")
        lib = ctypes.CDLL(path)
        for name, (argtypes, restype) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().ssm_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(t, name, dtypes, dev, ndim=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() not in ndim:
        raise ValueError("%s must have %s dims, got %d" % (name, ndim, t.dim()))


def ssm_scan_fwd(x, delta, A, B, C, D=None, y=None, **options):
    """Diagonal selective scan on the current CUDA stream; returns y (fp32),
    or (y, h_final) with ``return_final_state=True``."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    ins = (torch.float32, torch.bfloat16)
    for t, n in ((x, "x"), (delta, "delta"), (B, "B"), (C, "C")):
        _check(t, n, (x.dtype,) if x.dtype in ins else ins, dev, (3,))
    _check(A, "A", (torch.float32,), dev, (2,))
    _check(D, "D", (torch.float32,), dev, (1,))
    Bs, L, ED = x.shape
    N = A.shape[1]
    if delta.shape != x.shape or tuple(A.shape) != (ED, N) or tuple(B.shape) != (Bs, L, N) \
            or tuple(C.shape) != (Bs, L, N) or (D is not None and tuple(D.shape) != (ED,)):
        raise ValueError("shape mismatch: x, delta (Bs,L,ED); A (ED,N); B, C (Bs,L,N); D (ED)")
    if y is None:
        y = torch.empty((Bs, L, ED), dtype=torch.float32, device=dev)
    _check(y, "y", (torch.float32,), dev, (3,))
    bad = set(options) - set(_OPTION_KEYS)
    if bad:
        raise TypeError("unknown options: %s" % sorted(bad))
    if options:
        o, hf, keep = _options(x, ED, (Bs, ED, N), dev, **options)
        st = library().ssm_scan_fwd_ex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                       _ptr(y), Bs, L, ED, N, int(x.dtype == torch.bfloat16),
                                       ctypes.byref(o), _stream(dev))
        if st != 0:
            raise SsmError("ssm_scan_fwd_ex", st)
        return (y, hf) if options.get("return_final_state") else y
    name = "ssm_scan_fwd" if x.dtype == torch.float32 else "ssm_scan_fwd_bf16"
    fn = getattr(library(), name)
    st = fn(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y),
            Bs, L, ED, N, _stream(dev))
    if st != 0:
        raise SsmError(name, st)
    return y


def ssm_scan_fwd_bf16(x, delta, A, B, C, D=None, y=None, **options):
    """Same as ``ssm_scan_fwd`` but requires bf16 x, delta, B, C."""
    import torch
    if x.dtype != torch.bfloat16:
        raise TypeError("ssm_scan_fwd_bf16 takes bf16 x, delta, B, C")
    return ssm_scan_fwd(x, delta, A, B, C, D, y, **options)


def ssd_chunk_scan_fwd(x, dt, A_head, B, C, D=None, chunk: int = 256,
                       bidirectional: bool = False, y=None, **options):
    """Chunked scalar-decay scan on the current CUDA stream; returns y (fp32),
    or (y, h_final) with ``return_final_state=True``."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be bf16 or fp32")
    bf = (x.dtype,)
    _check(x, "x", bf, dev, (4,))
    _check(dt, "dt", bf, dev, (3,))
    _check(B, "B", bf, dev, (3, 4))
    _check(C, "C", bf, dev, (3, 4))
    _check(A_head, "A_head", (torch.float32,), dev, (1,))
    _check(D, "D", (torch.float32,), dev, (1,))
    Bs, L, H, P = x.shape
    G = B.shape[2] if B.dim() == 4 else 1
    if B.dim() == 4 and (C.dim() != 4 or C.shape[2] != G or H % G != 0):
        raise ValueError("B, C must be (Bs, L, G, N) with G dividing H")
    N = B.shape[-1]
    if tuple(dt.shape) != (Bs, L, H) or tuple(A_head.shape) != (H,) \
            or B.shape[0] != Bs or B.shape[1] != L or tuple(C.shape) != tuple(B.shape) \
            or (D is not None and tuple(D.shape) != (H,)):
        raise ValueError("shape mismatch: x (Bs,L,H,P); dt (Bs,L,H); A_head (H); B, C (Bs,L,[G,]N)")
    if y is None:
        y = torch.empty((Bs, L, H, P), dtype=torch.float32, device=dev)
    _check(y, "y", (torch.float32,), dev, (4,))
    bad = set(options) - set(_OPTION_KEYS)
    if bad:
        raise TypeError("unknown options: %s" % sorted(bad))
    if G > 1:
        options = dict(options, ngroups=G)
    if options or x.dtype != torch.bfloat16:
        o, hf, keep = _options(x, H, (Bs, H, P, N), dev, **options)
        st = library().ssd_chunk_scan_fwd_ex(_ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C),
                                             _ptr(D), _ptr(y), Bs, L, H, P, N, int(chunk),
                                             int(bool(bidirectional)),
                                             int(x.dtype == torch.bfloat16), ctypes.byref(o),
                                             _stream(dev))
        if st != 0:
            raise SsmError("ssd_chunk_scan_fwd_ex", st)
        return (y, hf) if options.get("return_final_state") else y
    st = library().ssd_chunk_scan_fwd(_ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C), _ptr(D),
                                      _ptr(y), Bs, L, H, P, N, int(chunk), int(bool(bidirectional)),
                                      _stream(dev))
    if st != 0:
        raise SsmError("ssd_chunk_scan_fwd", st)
    return y


def ssm_scan_bwd(x, delta, A, B, C, D, dy, **options):
    """Gradients of the diagonal scan for the upstream gradient dy (fp32,
    shaped like y): dict(dx, ddelta, dA, dB, dC, dD) as fp32 tensors (dD is
    None when D is None).  With the forward scan's options (dt_bias,
    dt_softplus, dt_limit, z, h0) the dict also holds dz, ddt_bias and dh0
    (None when the matching option is off), and ddelta is the gradient with
    respect to delta before the options."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    ins = (torch.float32, torch.bfloat16)
    for t, n in ((x, "x"), (delta, "delta"), (B, "B"), (C, "C")):
        _check(t, n, (x.dtype,) if x.dtype in ins else ins, dev, (3,))
    _check(A, "A", (torch.float32,), dev, (2,))
    _check(D, "D", (torch.float32,), dev, (1,))
    _check(dy, "dy", (torch.float32,), dev, (3,))
    Bs, L, ED = x.shape
    N = A.shape[1]
    if delta.shape != x.shape or dy.shape != x.shape or tuple(A.shape) != (ED, N) \
            or tuple(B.shape) != (Bs, L, N) or tuple(C.shape) != (Bs, L, N):
        raise ValueError("shape mismatch: x, delta, dy (Bs,L,ED); A (ED,N); B, C (Bs,L,N)")
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty((Bs, L, ED), **f32), ddelta=torch.empty((Bs, L, ED), **f32),
             dA=torch.empty((ED, N), **f32), dB=torch.empty((Bs, L, N), **f32),
             dC=torch.empty((Bs, L, N), **f32), dD=None if D is None else torch.empty(ED, **f32))
    bad = set(options) - (set(_OPTION_KEYS) - {"return_final_state"})
    if bad:
        raise TypeError("unknown options: %s" % sorted(bad))
    if options:
        o, _, keep = _options(x, ED, (Bs, ED, N), dev, **options)
        g["dz"] = torch.empty((Bs, L, ED), **f32) if options.get("z") is not None else None
        g["ddt_bias"] = torch.empty(ED, **f32) if options.get("dt_bias") is not None else None
        g["dh0"] = torch.empty((Bs, ED, N), **f32) if options.get("h0") is not None else None
        st = library().ssm_scan_bwd_ex(
            _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dy), _ptr(g["dx"]),
            _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
            _ptr(g["dz"]), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), Bs, L, ED, N,
            int(x.dtype == torch.bfloat16), ctypes.byref(o), _stream(dev))
        if st != 0:
            raise SsmError("ssm_scan_bwd_ex", st)
        return g
    st = library().ssm_scan_bwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dy),
                                _ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]),
                                _ptr(g["dC"]), _ptr(g["dD"]), Bs, L, ED, N,
                                int(x.dtype == torch.bfloat16), _stream(dev))
    if st != 0:
        raise SsmError("ssm_scan_bwd", st)
    return g


def ssd_chunk_scan_bwd(x, dt, A_head, B, C, D, dy, bidirectional: bool = False, **options):
    """Gradients of the chunked scan for the upstream gradient dy (fp32,
    shaped like y): dict(dx, ddt, dA, dB, dC, dD) as fp32 tensors (dB, dC
    shaped like B, C; dD is None when D is None).  With the forward scan's
    options (dt_bias, dt_softplus, dt_limit, z, h0) the dict also holds dz,
    ddt_bias and dh0 (None when the matching option is off), and ddt is the
    gradient with respect to dt before the options."""
    import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    ins = (torch.float32, torch.bfloat16)
    _check(x, "x", ins, dev, (4,))
    _check(dt, "dt", (x.dtype,), dev, (3,))
    _check(B, "B", (x.dtype,), dev, (3, 4))
    _check(C, "C", (x.dtype,), dev, (3, 4))
    _check(A_head, "A_head", (torch.float32,), dev, (1,))
    _check(D, "D", (torch.float32,), dev, (1,))
    _check(dy, "dy", (torch.float32,), dev, (4,))
    Bs, L, H, P = x.shape
    G = 1 if B.dim() == 3 else B.shape[2]
    N = B.shape[-1]
    bc = (Bs, L, N) if B.dim() == 3 else (Bs, L, G, N)
    if tuple(dt.shape) != (Bs, L, H) or tuple(A_head.shape) != (H,) or dy.shape != x.shape \
            or tuple(B.shape) != bc or tuple(C.shape) != bc:
        raise ValueError("shape mismatch: x, dy (Bs,L,H,P); dt (Bs,L,H); A_head (H); "
                         "B, C (Bs,L,N) or (Bs,L,G,N)")
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty((Bs, L, H, P), **f32), ddt=torch.empty((Bs, L, H), **f32),
             dA=torch.empty(H, **f32), dB=torch.empty(bc, **f32), dC=torch.empty(bc, **f32),
             dD=None if D is None else torch.empty(H, **f32))
    bad = set(options) - (set(_OPTION_KEYS) - {"return_final_state"})
    if bad:
        raise TypeError("unknown options: %s" % sorted(bad))
    if options:
        o, _, keep = _options(x, H, (Bs, H, P, N), dev, ngroups=G, **options)
        g["dz"] = torch.empty((Bs, L, H, P), **f32) if options.get("z") is not None else None
        g["ddt_bias"] = torch.empty(H, **f32) if options.get("dt_bias") is not None else None
        g["dh0"] = torch.empty((Bs, H, P, N), **f32) if options.get("h0") is not None else None
        st = library().ssd_chunk_scan_bwd_ex(
            _ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C), _ptr(D), _ptr(dy), _ptr(g["dx"]),
            _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
            _ptr(g["dz"]), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), Bs, L, H, P, N,
            int(bool(bidirectional)), int(x.dtype == torch.bfloat16), ctypes.byref(o),
            _stream(dev))
        if st != 0:
            raise SsmError("ssd_chunk_scan_bwd_ex", st)
        return g
    st = library().ssd_chunk_scan_bwd(
        _ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C), _ptr(D), _ptr(dy), _ptr(g["dx"]),
        _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
        Bs, L, H, P, N, G, int(bool(bidirectional)), int(x.dtype == torch.bfloat16), _stream(dev))
    if st != 0:
        raise SsmError("ssd_chunk_scan_bwd", st)
    return g


def ssm_scan_fwd_plan(Bs: int, L: int, ED: int, N: int, bf16: bool = True):
    """(states per thread, lanes per channel, time segments) the diagonal scan
    uses for this shape on the current device; time segments > 1 means two
    kernel launches per call."""
    s, g, k = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    st = library().ssm_scan_fwd_plan(Bs, L, ED, N, int(bool(bf16)), ctypes.byref(s),
                                     ctypes.byref(g), ctypes.byref(k))
    if st != 0:
        raise SsmError("ssm_scan_fwd_plan", st)
    return s.value, g.value, k.value


def ssm_check_device_errors(device=None) -> None:
    """Synchronise the current stream and raise SsmError if a kernel of the
    library abandoned its work after a bounded device wait ran out."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    st = library().ssm_check_device_errors(_stream(dev))
    if st != 0:
        raise SsmError("ssm_check_device_errors", st)


# ---- gated linear recurrence -----------------------------------------------------------
_BLOCK = 64      # SSM_GATED_BLOCK: steps between kept states; also columns that share an 8-bit scale
_CKPT8 = ("x_q", "r_q", "i_q", "x_s", "r_s", "i_s")


def _call(name, dev, *args):
    """Call a C entry point on the current stream of ``dev``.  These calls are
    short, so the marshalling is kept lean: addresses as integers, the
    stream's handle without a Stream object."""
    import torch
    index = dev.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(name, dev, *args)
    st = getattr(_lib or library(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise SsmError(name, st)


def _addr(t):
    return None if t is None else t.data_ptr()


def _fits(t, dtype, shape, dev):
    """The usual case of ``_check_shape``, without its messages."""
    return t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous()


def _saved_shapes(Bs, L, ED):
    q, s = (Bs, L, ED), (-(-ED // _BLOCK), Bs * L)
    return dict(states=(Bs, -(-L // _BLOCK), ED), x_q=q, r_q=q, i_q=q, x_s=s, r_s=s, i_s=s)


def _new_saved(save, Bs, L, ED, dev):
    """Empty tensors for what ``gated_scan_fwd`` keeps."""
    import torch
    shapes = _saved_shapes(Bs, L, ED)
    return {k: torch.empty(shapes[k], dtype=torch.int8 if k[1:] == "_q" else torch.float32, device=dev)
            for k in (("states",) if save == "states" else ("states",) + _CKPT8)}


def _saved_struct(saved):
    o = GatedSaved()
    for k, t in saved.items():
        setattr(o, k, t.data_ptr())
    return o


def _gated_inputs(x, gate_r, gate_i, lam, ndim):
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    if not x.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    _check(x, "x", (torch.bfloat16, torch.float32), dev, (ndim,))
    dtype, shape = x.dtype, x.shape
    for t, n in ((gate_r, "gate_r"), (gate_i, "gate_i")):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % n)
        if not _fits(t, dtype, shape, dev):
            _check_shape(t, n, (dtype,), dev, shape)
    if not isinstance(lam, torch.Tensor):
        raise TypeError("lam must be a torch.Tensor")
    if not _fits(lam, torch.float32, shape[-1:], dev):
        _check_shape(lam, "lam", (torch.float32,), dev, shape[-1:])
    return dev


def _check_shape(t, name, dtypes, dev, shape):
    if t is None:
        return
    _check(t, name, dtypes, dev)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def gated_scan_fwd(x, gate_r, gate_i, lam, c=8.0, reset=None, h0=None, return_final_state=False,
                   save=None, y=None):
    """Gated linear recurrence on the current CUDA stream:

        a_t = exp(-c softplus(lam) sigmoid(gate_r)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_i) x_t

    x, gate_r, gate_i: (Bs, L, ED) bf16 or fp32; lam: (ED) fp32; reset: (Bs, L)
    bool or uint8, true where a sequence starts (the state before it is
    dropped); h0: (Bs, ED) fp32.  Returns y (Bs, L, ED) in x's type; with
    ``return_final_state`` also h_final (Bs, ED) fp32; with ``save`` also the
    dict that ``gated_scan_bwd`` takes: ``save="states"`` keeps the state
    every 64 steps (the caller keeps x, gate_r, gate_i), ``save="8bit"`` also
    the 8-bit checkpoints of x, gate_r and gate_i in their place."""
    import torch
    dev = _gated_inputs(x, gate_r, gate_i, lam, 3)
    Bs, L, ED = x.shape
    _check_shape(reset, "reset", (torch.uint8, torch.bool), dev, (Bs, L))
    _check_shape(h0, "h0", (torch.float32,), dev, (Bs, ED))
    if save not in (None, "states", "8bit"):
        raise ValueError("save must be None, 'states' or '8bit'")
    if y is None:
        y = torch.empty_like(x)
    else:
        _check_shape(y, "y", (x.dtype,), dev, x.shape)
    hf = torch.empty((Bs, ED), dtype=torch.float32, device=dev) if return_final_state else None
    saved = _new_saved(save, Bs, L, ED, dev) if save is not None else None
    _call("gated_scan_fwd", dev, x.data_ptr(), gate_r.data_ptr(), gate_i.data_ptr(), lam.data_ptr(), c,
          _addr(reset), _addr(h0), y.data_ptr(), _addr(hf),
          None if saved is None else ctypes.byref(_saved_struct(saved)),
          Bs, L, ED, int(x.dtype == torch.bfloat16))
    out = (y,) + ((hf,) if return_final_state else ()) + ((saved,) if save is not None else ())
    return out if len(out) > 1 else y


def gated_scan_bwd(x, gate_r, gate_i, lam, dy, saved, c=8.0, reset=None, dh_final=None):
    """Gradients of ``gated_scan_fwd`` for dy (Bs, L, ED), of x's type:
    dict(dx, dgate_r, dgate_i) of dy's type, dlam (ED) and dh0 (Bs, ED) fp32.
    ``saved`` is the forward call's dict; where it holds the 8-bit checkpoints
    they are read in the place of x, gate_r and gate_i, which may be None.
    dh_final: (Bs, ED) fp32, the gradient with respect to the final state."""
    import torch
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    dev = dy.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(dy, "dy", (torch.bfloat16, torch.float32), dev, (3,))
    Bs, L, ED = dy.shape
    if not isinstance(saved, dict) or "states" not in saved or set(saved) not in (
            {"states"}, {"states", *_CKPT8}):
        raise ValueError("saved must be the dict of gated_scan_fwd(..., save='states' or '8bit')")
    if "x_q" in saved:
        x = gate_r = gate_i = None
        _check(lam, "lam", (torch.float32,), dev, (1,))
        if lam is None or lam.shape[0] != ED:
            raise ValueError("lam must have %d entries" % ED)
    else:
        if _gated_inputs(x, gate_r, gate_i, lam, 3) != dev:
            raise ValueError("x is on %s, expected %s" % (x.device, dev))
        if x.dtype != dy.dtype or x.shape != dy.shape:
            raise ValueError("dy must have the shape and type of x")
    shapes = _saved_shapes(Bs, L, ED)
    for k, t in saved.items():
        if t is None:
            raise ValueError("saved[%r] is missing" % k)
        dtype = torch.int8 if k[1:] == "_q" else torch.float32
        if not isinstance(t, torch.Tensor) or not _fits(t, dtype, shapes[k], dev):
            _check_shape(t, "saved[%r]" % k, (dtype,), dev, shapes[k])
    _check_shape(reset, "reset", (torch.uint8, torch.bool), dev, (Bs, L))
    _check_shape(dh_final, "dh_final", (torch.float32,), dev, (Bs, ED))
    g = {k: torch.empty_like(dy) for k in ("dx", "dgate_r", "dgate_i")}
    g["dlam"] = torch.empty(ED, dtype=torch.float32, device=dev)
    g["dh0"] = torch.empty((Bs, ED), dtype=torch.float32, device=dev)
    scratch = torch.empty(min(16, -(-L // _BLOCK)) * Bs * ED, dtype=torch.float32, device=dev)
    _call("gated_scan_bwd", dev, _addr(x), _addr(gate_r), _addr(gate_i), lam.data_ptr(), c, _addr(reset),
          dy.data_ptr(), _addr(dh_final), ctypes.byref(_saved_struct(saved)), g["dx"].data_ptr(),
          g["dgate_r"].data_ptr(), g["dgate_i"].data_ptr(), g["dlam"].data_ptr(), g["dh0"].data_ptr(),
          scratch.data_ptr(), Bs, L, ED, int(dy.dtype == torch.bfloat16))
    return g


def gated_scan_step(x, gate_r, gate_i, lam, states, pages=None, c=8.0, y=None):
    """One token of the gated recurrence for each row of a batch.
    x, gate_r, gate_i: (Bs, ED) bf16 or fp32; states: (num_pages, ED) fp32,
    updated in place at row b's page pages[b] ((Bs) int32; None: page b).  A
    row whose page lies outside the pool is idle: y is 0, no state changes.
    Returns y (Bs, ED) in x's type."""
    import torch
    dev = _gated_inputs(x, gate_r, gate_i, lam, 2)
    Bs, ED = x.shape
    if states is None:
        raise TypeError("states must be a torch.Tensor")
    _check(states, "states", (torch.float32,), dev, (2,))
    num_pages, columns = states.shape
    if columns != ED:
        raise ValueError("states must have %d columns" % ED)
    if pages is None:
        if num_pages < Bs:
            raise ValueError("states has fewer pages than x has rows")
    else:
        _check_shape(pages, "pages", (torch.int32,), dev, (Bs,))
    if y is None:
        y = torch.empty_like(x)
    else:
        _check_shape(y, "y", (x.dtype,), dev, x.shape)
    _call("gated_scan_step", dev, x.data_ptr(), gate_r.data_ptr(), gate_i.data_ptr(), lam.data_ptr(), c,
          states.data_ptr(), _addr(pages), y.data_ptr(), Bs, ED, num_pages, int(x.dtype is torch.bfloat16))
    return y


# ---- 8-bit activation checkpoints ------------------------------------------------------
def ckpt8_save(x):
    """(q, scale) of an activation tensor (bf16 or fp32, at least one
    dimension): q int8 shaped like x, scale fp32 (ceil(cols / 64), rows), where
    cols is x's last dimension and rows all others; 64 columns of a row share a
    scale."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(x, "x", (torch.bfloat16, torch.float32), dev)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    q = torch.empty(x.shape, dtype=torch.int8, device=dev)
    scale = torch.empty((-(-cols // _BLOCK), rows), dtype=torch.float32, device=dev)
    _call("ckpt8_save", dev, x.data_ptr(), q.data_ptr(), scale.data_ptr(), rows, cols, int(x.dtype == torch.bfloat16))
    return q, scale


def ckpt8_load(q, scale, dtype=None, out=None):
    """The values q * scale of ``ckpt8_save``'s result in ``dtype`` (bf16, the
    default, or fp32), shaped like q."""
    import torch
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(q, "q", (torch.int8,), dev)
    if q.dim() < 1:
        raise ValueError("q must have at least one dimension")
    cols = q.shape[-1]
    rows = q.numel() // cols if cols else 0
    if scale is None:
        raise TypeError("scale must be a torch.Tensor")
    _check_shape(scale, "scale", (torch.float32,), dev, (-(-cols // _BLOCK), rows))
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16 if dtype is None else dtype, device=dev)
    _check_shape(out, "out", (torch.bfloat16, torch.float32) if dtype is None else (dtype,), dev,
                 q.shape)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    _call("ckpt8_load", dev, q.data_ptr(), scale.data_ptr(), out.data_ptr(), rows, cols, int(out.dtype == torch.bfloat16))
    return out


# ---- pages of a state cache ------------------------------------------------------------
def _pool_sizes(pool, page_dim):
    """(device, layers, pages, bytes of a page of one layer) of a pool."""
    import torch
    if not isinstance(pool, torch.Tensor):
        raise TypeError("pool must be a torch.Tensor")
    if not pool.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    if not pool.is_contiguous():
        raise ValueError("pool must be contiguous")
    shape = pool.shape
    if not 0 <= page_dim < len(shape):
        raise ValueError("page_dim must name a dimension of pool")
    return (pool.device, math.prod(shape[:page_dim]), shape[page_dim],
            math.prod(shape[page_dim + 1:]) * pool.element_size())


def _page_list(t, name, dev):
    import torch
    if t is None:
        raise TypeError("%s must be a torch.Tensor" % name)
    _check(t, name, (torch.int32,), dev, (1,))


def _used(used, dev, num_pages):
    import torch
    if used is None:
        raise TypeError("used must be a torch.Tensor")
    _check_shape(used, "used", (torch.uint8, torch.bool), dev, (num_pages,))


def state_pages_fork(pool, used, src, page_dim=0):
    """Give each request of ``src`` (int32 page numbers; -1: a new sequence) a
    page of its own: the lowest free pages in the requests' order, with a copy
    of page src[k] of every layer, or zeros.  pool: (..., pages, ...) with its
    pages along ``page_dim``, the dimensions before it being layers; used:
    (pages) uint8 or bool, updated in place.  Returns the int32 page numbers,
    -1 where src[k] is not in use or no page was free."""
    import torch
    dev, layers, n_pages, size = _pool_sizes(pool, page_dim)
    _used(used, dev, n_pages)
    _page_list(src, "src", dev)
    dst = torch.empty_like(src)
    _call("state_pages_fork", dev, pool.data_ptr(), used.data_ptr(), src.data_ptr(), dst.data_ptr(), src.shape[0], layers,
          n_pages, size)
    return dst


def state_pages_copy(pool, src, dst, page_dim=0):
    """Copy page src[k] to page dst[k] of every layer (src[k] == -1: zeros).
    An entry with another page outside the pool is skipped.  No page may be
    written twice, or both read and written."""
    dev, layers, n_pages, size = _pool_sizes(pool, page_dim)
    _page_list(src, "src", dev)
    _page_list(dst, "dst", dev)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    _call("state_pages_copy", dev, pool.data_ptr(), src.data_ptr(), dst.data_ptr(), src.shape[0], layers, n_pages, size)


def state_pages_free(used, pages):
    """Mark the listed pages free; entries outside the pool are skipped."""
    import torch
    if not isinstance(used, torch.Tensor):
        raise TypeError("used must be a torch.Tensor")
    dev = used.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(used, "used", (torch.uint8, torch.bool), dev, (1,))
    _page_list(pages, "pages", dev)
    _call("state_pages_free", dev, used.data_ptr(), pages.data_ptr(), pages.shape[0], used.shape[0])


def state_pages_compact(pool, used, pages=None, page_dim=0):
    """Move the pages in use to the front of the pool: the j-th one at or
    above their number goes to the j-th free page below it, the others stay.
    used is updated in place, and so is ``pages``, a list of page numbers
    (negative entries stay, pages not in use become -1).  Returns each page's
    new number ((pages) int32, -1 for a free page)."""
    import torch
    dev, layers, n_pages, size = _pool_sizes(pool, page_dim)
    _used(used, dev, n_pages)
    if pages is not None:
        _page_list(pages, "pages", dev)
    moved = torch.empty(n_pages, dtype=torch.int32, device=dev)
    scratch = torch.empty(2 * n_pages + 2, dtype=torch.int32, device=dev)
    _call("state_pages_compact", dev, pool.data_ptr(), used.data_ptr(), moved.data_ptr(), _addr(pages),
          scratch.data_ptr(),
          0 if pages is None else pages.shape[0], layers, n_pages, size)
    return moved
