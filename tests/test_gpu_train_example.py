"""examples/train_adapters.py: the layer, the loss, the gradients and the
update together.  Plain descent on a fixed batch: the loss starts near the
loss of a uniform guess and must fall well below it; without one of the parts
(say, gradients of the wrong sign) it does not fall at all."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("train_adapters",
                                                  os.path.join(ROOT, "examples", "train_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("rank", [16, 64])
def test_the_loss_falls(rank):
    vocab = 1000
    history = _example().train(steps=30, tokens=256, hidden=256, vocab=vocab, rank=rank, loras=3)
    assert all(math.isfinite(v) for v in history)
    assert abs(history[0] - math.log(vocab)) < 3.0
    assert history[-1] < 0.5 * history[0], history


def test_steps_repeat():
    mod = _example()
    a = mod.train(steps=5, tokens=100, hidden=128, vocab=333, rank=8, loras=2)
    b = mod.train(steps=5, tokens=100, hidden=128, vocab=333, rank=8, loras=2)
    assert a == b
