"""The serving example with its latents in 8 bits: what the cache holds is read back and attended to; the tolerance is that of the
bf16 cache (tests/test_gpu_latent_example.py), since the 64-bit form works on the rows that were read back."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_serves_from_8_bit_pages_and_agrees():
    spec = importlib.util.spec_from_file_location("latent_serving", os.path.join(ROOT, "examples", "latent_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(0, eight=True) <= 6 * 2.0 ** -8
    assert example.main(1, eight=True) <= 6 * 2.0 ** -8
