"""The operators together, as examples/policy_gradient.py uses them: the policy
learns its task (by chance it is right one time in 64), the same on every run."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "policy_gradient.py")


def test_policy_learns_its_task():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("policy_gradient", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last = example.train(300, log=None)
    assert first < 0.1
    assert last > 0.5
    assert example.train(20, log=None) == example.train(20, log=None)
