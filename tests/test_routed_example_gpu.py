"""The routed products in one block: it trains, and it decodes what torch computes."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "routed_layer.py")


def test_example_trains_and_decodes():
    spec = importlib.util.spec_from_file_location("routed_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, error = example.main(["--steps", "30", "--tokens", "256", "--hidden", "128", "--inner", "64"])
    assert losses[-1] < 0.9 * losses[0]
    assert all(b < a + 1e-3 for a, b in zip(losses, losses[1:]))
    # the block rounds its projection, inner rows and output to bf16: three errors of 2^-8 at most
    assert error < 3 * 2.0 ** -8
