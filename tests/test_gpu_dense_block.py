"""The example that trains a pre-norm dense block and serves it on mx8 weights."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_example_trains_and_serves():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_block.py")
    spec = importlib.util.spec_from_file_location("dense_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, w = ex.train(256, 512, 100, 15)
    assert losses[-1] < 0.9 * losses[0]
    assert all(b < a for a, b in zip(losses, losses[1:]))
    off = ex.serve(w, 100)
    # x, weights and act(gate) * up each carry e4m3's rounding, 2^-4 at most and ~2.6% as a root mean square: five of
    # them (both operands of three products) add up to ~6%
    assert set(off) == {1, 100} and all(0.0 < v < 0.12 for v in off.values())
