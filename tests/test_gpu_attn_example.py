"""The example runs, and its outputs are as near to plain attention as 8-bit keys and values allow."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_example_attention_layer_runs():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # A held value is off by at most 2^-4 of itself, evenly spread: 2^-4 / sqrt(3) = 0.036 in root mean square.
    # That much of a value goes to the outputs as it is. Of a key, it moves a score q k / sqrt(128) of normal
    # numbers by 0.036 in root mean square, and the weight by as much of itself. Both together: 0.051 of the
    # outputs, whose weighted sums take signal and errors alike; q and the weights in bf16 add under 0.004.
    # Twice that covers how far a step of two rows may lie from its mean.
    assert m.main() < 0.11
