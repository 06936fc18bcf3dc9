"""A layer trained with 8-bit products and the orthogonalised update: it runs, and its gradients are right."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "scaled_layer.py")


def test_example_runs_and_its_gradients_are_right():
    spec = importlib.util.spec_from_file_location("scaled_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, errors = example.main(["--steps", "6", "--tokens", "200", "--inputs", "264", "--outputs", "136"])
    assert len(losses) == 6 and all(math.isfinite(v) for v in losses)
    # y and dx are rounded to bf16, half a step of 2^-8 an element at most; dw is fp32: its sums' rounding, at most
    # (128 + 2 + 4) steps of 2^-23 of the sum of magnitudes, which random signs make up to sqrt(200) of the norm
    assert errors[0] <= 2.0 ** -8 + 1e-5 and errors[1] <= 2.0 ** -8 + 1e-5
    assert errors[2] <= 134 * 2.0 ** -23 * 200 ** 0.5
