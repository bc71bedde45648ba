"""Clipping where the norm, or the factor, leaves float32's range.

A value is off by its products' rounding to float32 (2^-24), the factor's where it is a float32
(2^-24) and its own rounding (half a step of its type)."""
import math

import pytest
import torch

from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


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


@pytest.mark.parametrize("max_norm", [2.0, 1e-3, 1e-6, 1e-20, 0.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_factors_below_the_normal_numbers(dtype, max_norm):
    """Norms of about 2.3e38: the factors lie around and below 2^-126, the results do not."""
    gen = torch.Generator().manual_seed(1)
    big = (torch.rand(1000, generator=gen) * 2e37 - 1e37).to(dtype)
    ts = [torch.tensor([2e38, 1e38, -3e37], device=DEV).to(dtype), big.to(DEV)]
    before = [t.clone() for t in ts]
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))
    assert norm < 3.4e38
    got = ssd.clip_grads(ts, max_norm)
    assert abs(float(got) - norm) <= 2.0 ** -23 * norm
    for a, b in zip(before, ts):
        want = a.double() * (max_norm / norm)
        assert ((b.double() - want).abs() <= (HALF[dtype] + 3 * 2.0 ** -24) * want.abs()).all()
