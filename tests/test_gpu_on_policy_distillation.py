"""The example that runs sampling, scoring and distillation together: the loss falls, and two
runs give the same tokens and weights bit for bit."""
import importlib.util
import os

import pytest
import torch

from helpers import bits_equal, cuda_or_skip

pytestmark = pytest.mark.gpu


def test_example():
    cuda_or_skip()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "on_policy_distillation.py")
    spec = importlib.util.spec_from_file_location("on_policy_distillation", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, token, weight = example.train(steps=5, rows=200, hidden=128, vocab=3001, slots=16)
    again = example.train(steps=5, rows=200, hidden=128, vocab=3001, slots=16)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert losses == again[0] and torch.equal(token, again[1]) and bits_equal(weight, again[2])
    assert ((token >= 0) & (token < 3001)).all()
