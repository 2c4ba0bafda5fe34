"""GPU test of examples/low_bit_linear.py: trained with an 8-bit saved input, served in 4 bits."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_trains_and_serves():
    spec = importlib.util.spec_from_file_location(
        "low_bit_linear", os.path.join(ROOT, "examples", "low_bit_linear.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, away, apart = example.main(1000, 264, 130, 40)
    # A step of 0.5 on the mean squared error of unit inputs halves the error of each
    # weight or better, less what 2-byte inputs and gradients lose.
    assert losses[-1] < 1e-3 * losses[0]
    # 4 bits: steps of a range of some six deviations over 15, so an error of a step
    # over sqrt(12): 0.12 of a deviation.
    assert away < 0.2
    # Two kernels, the same stored weight: fp32 sums of 264 products.
    assert apart < 264 * 2.0 ** -22
