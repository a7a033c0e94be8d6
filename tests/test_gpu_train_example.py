"""The example that runs the training-head operators together with the
optimizer step: both models learn."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_train_head_example_learns():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("train_head", os.path.join(ROOT, "examples", "train_head.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    teacher, student = mod.train(steps=300)
    # 1003 tokens with four equally likely successors each: from about ln 1003 = 6.9 towards ln 4 = 1.4
    assert teacher[0] > 5.0 and teacher[1] < 3.0, teacher
    assert student[1] < 0.5 * student[0], student
