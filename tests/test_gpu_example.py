"""The example that trains a cross attention on transport plans runs as it is documented."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_distil_plan_learns_and_answers_point_by_point():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "distill_plan.py")
    spec = importlib.util.spec_from_file_location("distill_plan", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, apart = example.main(steps=120, report=False)
    assert last < 0.2 * first
    # both outputs are bfloat16 of values below about 4, summed over 512 inputs of `o`
    assert apart < 0.05
