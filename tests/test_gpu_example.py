"""The serving example runs and its attention outputs agree with plain attention: within half a bf16 step (2^-8) of the
largest output, its weights' f16 rounding (2^-11) and a margin of two for the accumulated value weights."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_hybrid_serving_example():
    spec = importlib.util.spec_from_file_location("hybrid_serving", os.path.join(ROOT, "examples", "hybrid_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main() <= 2.0 ** -8 + 2 * 2.0 ** -11
    assert mod.main(prompts=(1, 63, 64, 65), steps=3, seed=1) <= 2.0 ** -8 + 2 * 2.0 ** -11
