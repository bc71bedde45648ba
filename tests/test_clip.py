"""The norm over many tensors and clipping (grad_norm, clip_grads) against float64.

Bounds: squares and sums are float64, so the norm is off by its own rounding to float32 (2^-24)
and the factor by 2^-24; a value is off by the factor's rounding, the product's (2^-24 each) and
its own (half a step of its type)."""
import math

import pytest
import torch

from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(sizes, seed=0, dtypes=(torch.float32, torch.bfloat16), std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * std * 10.0 ** -(k % 3)).to(dtypes[k % len(dtypes)]).to(DEV)
            for k, n in enumerate(sizes)]


def norm_of(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def check(before, after, got, max_norm):
    ref = norm_of(before)
    assert got.dtype == torch.float32 and got.shape == ()
    assert abs(float(got) - ref) <= 2.0 ** -23 * ref
    f = min(1.0, max_norm / ref) if ref > 0 else 1.0
    for a, b in zip(before, after):
        want = a.double() * f
        if f == 1.0:
            assert torch.equal(a, b)
        else:
            assert ((b.double() - want).abs() <= (HALF[a.dtype] + 3 * 2.0 ** -24) * want.abs() + 2.0 ** -133).all()


SIZES = {
    "one": [1], "two odd": [3, 5], "empty among others": [0, 7, 0], "all empty": [0, 0], "a block": [64, 4096, 63, 4097, 100000],
    "large": [5000000, 17, 3000001], "many": [1 + (37 * i) % 501 for i in range(400)], "single launch full": [8] * 128,
    "one more": [8] * 129,
}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("over", [0.3, 3.0])
def test_in_place_and_out(sizes, over):
    ts = make(SIZES[sizes], seed=1)
    max_norm = max(norm_of(ts) * over, 1e-3)
    before = [t.clone() for t in ts]
    assert torch.equal(ssd.grad_norm(ts), ssd.clip_grads(ts, max_norm, out=(out := [torch.full_like(t, 7.0) for t in ts])))
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    check(before, out, ssd.grad_norm(ts), max_norm)
    versions = [t._version for t in ts]
    got = ssd.clip_grads(ts, max_norm)
    check(before, ts, got, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(ts, out))
    assert all(t._version > v for t, v in zip(ts, versions))


def test_starts_off_16_bytes():
    """Views that begin at every element of 16 bytes, in and out differently."""
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.randn(40000, device=DEV).to(dtype)
        dst = torch.zeros(40000, device=DEV, dtype=dtype)
        ins = [buf[1000 * i + i: 1000 * i + i + 900 + i] for i in range(16)]
        for shift in (0, 1, 5):
            outs = [dst[1000 * i + i + shift: 1000 * i + i + shift + 900 + i] for i in range(16)]
            dst.zero_()
            got = ssd.clip_grads(ins, 2.0, out=outs)
            check(ins, outs, got, 2.0)
            touched = torch.zeros_like(dst, dtype=torch.bool)
            for i in range(16):
                touched[1000 * i + i + shift: 1000 * i + i + shift + 900 + i] = True
            assert float(dst[~touched].abs().max()) == 0.0


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(value):
    ts = make([100, 5000, 3])
    ts[1][77] = value
    before = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts]
    n = ssd.clip_grads(ts, 1.0, out=out)
    assert not math.isfinite(float(n))
    ssd.clip_grads(ts, 1.0)
    for a, b, c in zip(before, ts, out):
        assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) and torch.equal(a.nan_to_num(5.0), c.nan_to_num(5.0))


def test_squares_beyond_float32():
    ts = [torch.tensor([3e30, -4e30], device=DEV), torch.tensor([1e-30, 0.0], device=DEV, dtype=torch.bfloat16)]
    before = [t.clone() for t in ts]
    check(before, ts, ssd.clip_grads(ts, 1.0), 1.0)
    ts = [torch.tensor([3e-30, 4e-30], device=DEV)]
    n = ssd.grad_norm(ts)
    assert abs(float(n) / 5e-30 - 1) < 2.0 ** -22
    assert abs(float(ssd.clip_grads(ts, 1e-31)) / 5e-30 - 1) < 2.0 ** -22 and abs(float(ts[0][0]) / 6e-32 - 1) < 1e-6


def test_limits():
    ts = make([300, 20])
    before = [t.clone() for t in ts]
    ssd.clip_grads(ts, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    ssd.clip_grads(ts, 0.0)
    assert all(float(t.abs().max()) == 0.0 for t in ts)
    zeros = [torch.zeros(50, device=DEV)]
    assert float(ssd.clip_grads(zeros, 1.0)) == 0.0 and float(zeros[0].abs().max()) == 0.0


def test_same_order_every_time():
    ts = make([1000003, 77, 400000], seed=4)
    n = ssd.grad_norm(ts)
    assert all(torch.equal(ssd.grad_norm(ts), n) for _ in range(5))


def test_shapes_of_any_rank():
    ts = [torch.randn(3, 4, 5, device=DEV), torch.randn((), device=DEV), torch.randn(2, 0, device=DEV)]
    before = [t.clone() for t in ts]
    check(before, ts, ssd.clip_grads(ts, 0.5), 0.5)
