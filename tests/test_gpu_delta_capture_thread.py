"""A call that a host thread which has made no other yet records into a graph
that another thread captures."""
import threading

import pytest
import torch

import linear_recurrence_ssm_gb300 as lrs
from delta_calls import at, sizes
from test_gpu_delta import BF, cuda, inputs

pytestmark = pytest.mark.gpu


def test_a_new_thread_s_call_while_a_graph_is_captured(cuda_device):
    i, _ = inputs(1, 1, 200, 1, 2, 64, 64, BF)
    c = cuda(i, cuda_device)
    want = lrs.delta_rule_fwd(**c, scale=1.0)
    size = sizes(c, 0)
    lib = lrs.library()
    y, scratch = torch.zeros_like(want), torch.empty(lib.delta_rule_fwd_scratch(*size), dtype=torch.uint8, device=cuda_device)
    graph, got, stream = torch.cuda.CUDAGraph(), [], torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        got.append(lib.delta_rule_fwd(*(at(c[w]) for w in ("q", "k", "v", "g", "beta")), 1.0, None, None, at(y), None, None,
                                      None, at(scratch), *size, stream.cuda_stream))

    with torch.cuda.graph(graph, stream=stream):
        thread = threading.Thread(target=call)
        thread.start()
        thread.join()
    assert got == [0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
