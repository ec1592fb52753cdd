"""The fine-tuning example: the losses and the optimizer step used together."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_lowers_each_loss():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_efficient_optimizer_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("finetune_losses", os.path.join(ROOT, "examples", "finetune_losses.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out = example.main(["--vocab", "4003", "--width", "64", "--batch", "4", "--length", "32", "--steps", "8"])
    assert all(math.isfinite(v) for losses in out.values() for v in losses)
    assert out["distill"][-1] < out["distill"][0]
    # a model that prefers neither sequence has ln 2
    assert abs(out["preference"][0] - math.log(2)) < 1e-3 and out["preference"][-1] < out["preference"][0]
    # within four steps on the same samples
    assert out["policy"][3] < out["policy"][0]
