"""The example that trains a block with a memory layer: what a step does to the parameters, whose gradients
test_gpu_training_step.py compares with autograd's."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "train_block.py")


def test_every_parameter_moves_against_its_gradient(monkeypatch):
    spec = importlib.util.spec_from_file_location("train_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    seen = []  # parameters and gradients ahead of each step: the gradients are those of the step before

    class Kept(example.Block):
        def lowered(self):
            seen.append(tuple({n: t.clone() for n, t in d.items()} for d in (self.params, self.grads)))
            return super().lowered()
    monkeypatch.setattr(example, "Block", Kept)
    rate = 0.5
    example.train(steps=3, rate=rate, B=130)
    assert len(seen) == 3
    for (before, _), (after, grads) in zip(seen, seen[1:]):
        for name in before:
            if name == "norm1":
                assert torch.equal(after[name], before[name])
                continue
            assert bool((grads[name] != 0).any()), name
            assert torch.equal(after[name], before[name].sub(grads[name], alpha=rate)), name
            assert not torch.equal(after[name], before[name]), name
