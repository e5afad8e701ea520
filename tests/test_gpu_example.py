"""The example that trains a feed-forward block and a memory layer from a teacher's top logits."""
import importlib.util
import math
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "distill_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("distill_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("B", [300, 40])
def test_the_loss_falls(example, B):
    losses = example.train(steps=12, B=B)
    assert all(math.isfinite(v) for v in losses)
    # (full-batch gradient steps of a size that a few steps more than halve the loss with)
    assert losses[-1] < 0.8 * losses[0]
    assert min(losses) == pytest.approx(min(losses[-4:]))
