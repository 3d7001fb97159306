"""The example runs the operators together: a predictor learns, its beam search
answers with codes that decode, and beams encode better than single codes."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_code_predictor_example():
    spec = importlib.util.spec_from_file_location("code_predictor", os.path.join(ROOT, "examples", "code_predictor.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, greedy, predicted, searched = example.main(["--frames", "500", "--steps", "30"])
    assert all(math.isfinite(v) for v in losses) and losses[-1] < losses[0]
    assert math.isfinite(predicted)
    # one code at a time is one of the paths that wider beams may keep: they end nearer to the frames
    assert searched < greedy
