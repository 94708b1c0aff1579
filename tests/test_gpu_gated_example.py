"""The example around the gated recurrence (GPU): it learns, and its served
tokens are those of whole scans."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_recurrence.py")


def test_example_trains_and_serves(cuda_device):
    spec = importlib.util.spec_from_file_location("gated_recurrence_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer = m.Layer(8, 128)
    losses = m.train(layer, 8, 60, Bs=4, L=100)
    # running averages of white noise: predicting 0 costs their variance,
    # (1 - 0.95)^2 / (1 - 0.95^2) = 0.026 late in the sequence; the start is
    # a random layer's O(1)
    assert losses[-1] < 0.2 * losses[0], (losses[0], losses[-1])
    # h is rounded to bf16 in either way (2^-9 of it, 2^-8 where the two
    # round apart), and summed over 128 channels with weights of 1/sqrt(128):
    # 2^-8 sqrt(128) max|h| / sqrt(128) with max|h| < 8
    assert m.serve(layer, 8) < 8 * 2.0 ** -8
