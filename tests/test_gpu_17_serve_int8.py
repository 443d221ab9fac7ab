"""The int8 operators together: the example layer against fp32."""
import importlib.util
import os

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_attention_layer(gpu):
    """Roundings to 127 levels of a row's (a block's, an output channel's) largest value. For normal values the largest of
    n is about sqrt(2 ln 2n) standard deviations: 4.0 of 1024 and up to 4.9 of a cache block's 8192, so a rounding is off
    by 4.9 / (127 sqrt 12) = 1.1% at most (rms). In line: activations, weights and v in the cache (3 of them before the
    softmax's average, which keeps relative errors of independent values), activations and weights of o: sqrt(5) 1.1%;
    errors of q.k are of 1 / 40 of a score's deviation and add a like amount; bf16 between the steps 0.2% each. Together
    below 4%."""
    announce("attention layer in 8 bits, prompts and decoded tokens")
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "attention_layer_int8.py")
    spec = importlib.util.spec_from_file_location("attention_layer_int8", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, later = example.run(gpu)
    assert first < 0.04 and later < 0.04, (first, later)
