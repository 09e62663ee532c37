"""The feed-forward example trains, and its 4-bit form answers alike."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_feed_forward_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out = mod.main(hidden=512, inner=1024, tokens=1024, steps=20)
    assert out["losses"][-1] < 0.75 * out["losses"][0]
    # 4-bit steps of a group of normal weights are about 0.4 standard deviations wide:
    # an error of 0.4 / sqrt(12) = 0.12 per product, three of which meet
    assert 0 < out["error"] < 0.35
