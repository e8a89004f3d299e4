"""examples/sharded_step.py: weights that do not split evenly over the ranks are
refused before anything is made of them (needs no GPU)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sharded_step", os.path.join(ROOT, "examples", "sharded_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("world,width", [(3, 256), (5, 96), (7, 8), (2, 1)])
def test_a_width_that_does_not_divide(example, world, width):
    with pytest.raises(ValueError, match="divide"):
        example.Step(world, width=width)
