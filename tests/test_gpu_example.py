"""The operators together, as the example runs them: an 8-bit layer, the
distillation loss, the layer's gradient, the compressor."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("distill_int8", os.path.join(ROOT, "examples", "distill_int8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_a_student_learns_through_compressed_gradients():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    losses, bits = _example().train(steps=40, batch=128, width=256, vocab=1000, top=16, bucket=512, levels=16)
    print(losses[0], losses[-1], bits)
    assert all(l == l for l in losses)
    # the mean of the last five steps is well below the start, for gradients of a few bits
    assert sum(losses[-5:]) / 5 < 0.7 * losses[0]
    assert bits < 8
