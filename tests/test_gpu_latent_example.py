"""The serving example: prompts, parallel samples, generation, rollback, end and packing through the
library's calls, every attention output against the 64-bit form on the request's own tokens.

The form it is checked against expands the stored latents to bf16 keys and values as the prefill
does; the absorbed form rounds the absorbed query and its latent output instead.  Each of those
roundings is within 2^-8 of a value of the outputs' size times the few sums it enters: 6 * 2^-8
bounds them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_serves_and_agrees():
    spec = importlib.util.spec_from_file_location("latent_serving", os.path.join(ROOT, "examples", "latent_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(0) <= 6 * 2.0 ** -8
    assert example.main(1) <= 6 * 2.0 ** -8
