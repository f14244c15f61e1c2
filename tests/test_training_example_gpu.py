"""The training example runs the expert products, the head's loss and all their gradients together: the loss starts
where an untrained head's does and falls as the model learns its task."""
import math
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_the_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import expert_head_training as example
    finally:
        sys.path.pop(0)
    losses = example.train(steps=40, vocab=1000, hidden=256, tokens=1024, log=lambda *_: None)
    assert math.log(1000) < losses[0] < math.log(1000) + 3
    assert losses[-1] < 0.2 * losses[0]
