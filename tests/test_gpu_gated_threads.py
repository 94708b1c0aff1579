"""Gated calls from several host threads at once."""
import ctypes
import threading

import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs

pytestmark = pytest.mark.gpu
ED = 64


class Work:
    """Forward and gradients of one sequence through the C entry points, on a
    stream of its own: a loop of calls is in the library most of its time."""

    def __init__(self, L, dtype, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        self.x, self.r, self.i, self.dy = (torch.randn(1, L, ED, generator=g, device=device).to(dtype)
                                           for _ in range(4))
        self.lam = torch.full((ED,), -4.0, device=device)
        self.y, self.dx, self.dr, self.di = (torch.empty_like(self.x) for _ in range(4))
        self.dlam, self.states = torch.empty_like(self.lam), torch.empty(1, -(-L // 64), ED, device=device)
        self.scratch = torch.empty(16 * ED, device=device)
        self.saved = lrs.GatedSaved()
        self.saved.states = self.states.data_ptr()
        self.stream = torch.cuda.Stream(device)
        torch.cuda.synchronize(device)
        lib, at = lrs.library(), [t.data_ptr() for t in (self.x, self.r, self.i, self.lam)]
        sizes = (1, L, ED, int(dtype == torch.bfloat16), self.stream.cuda_stream)
        self.fwd = lib.gated_scan_fwd, (*at, 8.0, None, None, self.y.data_ptr(), None,
                                        ctypes.byref(self.saved), *sizes)
        self.bwd = lib.gated_scan_bwd, (*at, 8.0, None, self.dy.data_ptr(), None, ctypes.byref(self.saved),
                                        *(t.data_ptr() for t in (self.dx, self.dr, self.di, self.dlam)), None,
                                        self.scratch.data_ptr(), *sizes)

    def outputs(self):
        self.stream.synchronize()
        return [t.clone() for t in (self.y, self.states, self.dx, self.dr, self.di, self.dlam)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sequences_of_different_lengths(cuda_device, dtype):
    """A kernel takes more shared memory the more blocks share a sequence.
    Calls that differ in that do not disturb each other: none fails, and the
    results are those of calls made one after another."""
    works = [Work(L, dtype, cuda_device, seed=L) for L in (1, 2100, 64, 1300, 300, 30)]
    start, failed = threading.Barrier(len(works)), []

    def thread(w):
        torch.cuda.set_device(cuda_device)
        start.wait()
        for _ in range(3000):
            for call, args in (w.fwd, w.bwd):
                status = call(*args)
                if status != 0:
                    failed.append(status)

    threads = [threading.Thread(target=thread, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    at_once = [w.outputs() for w in works]
    assert failed == []
    for w, got in zip(works, at_once):
        for call, args in (w.fwd, w.bwd):
            assert call(*args) == 0
        for a, b in zip(got, w.outputs()):
            assert torch.equal(a, b)
