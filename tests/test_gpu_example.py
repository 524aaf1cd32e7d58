"""The example that uses the matrix step, layer norm and AdamW together: it
learns, and it gives the same losses every time."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("width,hidden,world", [(256, 1024, 4), (64, 96, 2)])
def test_example_learns_and_repeats(width, hidden, world):
    """The target's part beyond x has a mean square of about 0.39 (tanh of a
    unit normal); a block that learns it leaves well under half after 60
    steps, and one that does not stays there."""
    mod = load()
    first = mod.train(width, hidden, world, steps=60, rows=256)
    assert 0.3 < first[0] < 0.6
    assert sum(first[-5:]) / 5 < 0.5 * first[0]
    assert mod.train(width, hidden, world, steps=60, rows=256) == first
