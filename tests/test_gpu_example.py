"""The example of an expert layer runs, learns and serves."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_expert_layer_example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, off = m.main(40)
    # zero weights start at the teacher's own power, 1
    assert 0.8 < losses[0] < 1.2 and losses[-1] < 0.5 * losses[0]
    assert off < 0.8
