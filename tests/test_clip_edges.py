"""Clipping where the norm leaves float32's range."""
import math

import pytest
import torch

from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 0.0])
def test_a_norm_beyond_float32_changes_nothing(max_norm):
    """The norm that the caller receives is infinite, though no element is."""
    ts = [torch.tensor([3e38, -3e38], device=DEV), torch.tensor([1.0, 3e38], device=DEV, dtype=torch.bfloat16)]
    before = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts]
    assert math.isinf(float(ssd.clip_grads(ts, max_norm, out=out)))
    assert all(torch.equal(a, b) for a, b in zip(before, out))
    assert math.isinf(float(ssd.clip_grads(ts, max_norm)))
    assert all(torch.equal(a, b) for a, b in zip(before, ts))
