"""Layer norm (norm_fwd, norm_bwd) against float64.

Tolerance: means and variances are sums of D float32 terms in runs of at most 32 per lane and
a tree across lanes: 40 * 2^-24 of the terms' sizes, a few more for rstd and the products;
with rows whose mean is a few standard deviations that stays below 2e-5 of the largest
value.  Sums over rows: running sums of at most rows / 512 (or rows) terms: 1e-4."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL, TOL_SUM = 2e-5, 1e-4

SHAPES = [  # rows, D, elements from row to row beyond D
    (1, 1, 0), (1, 768, 0), (3, 2, 0), (2, 63, 1), (5, 64, 0), (4, 65, 3), (7, 255, 0), (6, 257, 0), (9, 512, 8),
    (3, 520, 0), (1000, 1024, 0), (11, 1025, 0), (5, 2048, 2048), (3, 2056, 0), (2, 4095, 0), (4, 4096, 0), (3, 8192, 0),
    (2, 8199, 0), (3, 16384, 0), (2, 32776, 0), (1500, 40, 0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("affine", [True, False])
def test_forward_and_backward(shape, dtype, affine):
    rows, D, extra = shape
    gen = torch.Generator().manual_seed(rows + D)
    full = (torch.randn(rows, D + extra, generator=gen) * 2 + 1.5).to(dtype)
    x = full[:, :D]
    dy = torch.randn(rows, D, generator=gen).to(dtype)
    w = 1 + 0.3 * torch.randn(D, generator=gen) if affine else None
    b = torch.randn(D, generator=gen) if affine else None
    dev = lambda t: None if t is None else t.to(DEV)
    xg = full.to(DEV)[:, :D]
    y, mean, rstd = ssd.norm_fwd(xg, dev(w), dev(b), want_stats=True)
    y2 = ssd.norm_fwd(xg, dev(w), dev(b))
    g = ssd.norm_bwd(dev(dy), xg, dev(w), mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    xr, wr, br = R.up(x).requires_grad_(True), R.up(w), R.up(b)
    one = torch.ones(D, dtype=R.F64) if wr is None else wr
    zero = torch.zeros(D, dtype=R.F64) if br is None else br
    one.requires_grad_(True)
    zero.requires_grad_(True)
    yr, mr, rr = R.norm(xr, one, zero)
    dx, dw, db = R.grads((yr,), (R.up(dy),), [xr, one, zero])
    R.check(y, yr, dtype, TOL, "y")
    R.check(mean, mr, torch.float32, TOL, "mean")
    R.check(rstd, rr, torch.float32, TOL, "rstd")
    # with one or two channels the terms of dx, of size rstd |dy w|, cancel in every element
    R.check(g.dx, dx, dtype, TOL, "dx", scale=float((rr.detach()[:, None] * R.up(dy) * one.detach()).abs().max()))
    R.check(g.dweight, dw, torch.float32, TOL_SUM, "dweight", scale=float(R.up(dy).abs().max()))
    R.check(g.dbias, db, torch.float32, TOL_SUM, "dbias")


def test_rows_of_one_value_and_large_offsets():
    """A constant row has variance 0 (y = bias); an offset of 1e3 standard deviations costs
    the offset's own rounding (1e3 * 2^-24), not its square."""
    D = 777
    x = torch.randn(4, D, generator=torch.Generator().manual_seed(0))
    x[0] = 3.25
    x[1] = 0.0
    x[2] += 1000.0
    w, b = torch.rand(D) + 0.5, torch.randn(D)
    y = ssd.norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    torch.cuda.synchronize()
    yr, _, _ = R.norm(R.up(x), R.up(w), R.up(b))
    R.check(y[:2], yr[:2], torch.float32, TOL, "constant rows")
    R.check(y[2:3], yr[2:3], torch.float32, 3e-4, "large offset")
    R.check(y[3:], yr[3:], torch.float32, TOL, "ordinary row")


def test_gradient_against_differences():
    """Central differences with a step of 1e-2 on rows of spread 2: truncation (5e-3)^2 and
    rounding 1e-6 / 1e-2 stay below 1e-3."""
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(6, 300, generator=gen) * 2).to(DEV), torch.randn(6, 300, generator=gen).to(DEV)
    w, b = (1 + 0.2 * torch.randn(300, generator=gen)).to(DEV), torch.randn(300, generator=gen).to(DEV)
    _, mean, rstd = ssd.norm_fwd(x, w, b, want_stats=True)
    g = ssd.norm_bwd(dy, x, w, mean, rstd)
    for k, grad in enumerate(g):
        args = [x, w, b]
        v = torch.randn(args[k].shape, generator=gen).to(DEV)

        def loss(s):
            e = list(args)
            e[k] = args[k] + s * v
            return float((ssd.norm_fwd(*e).double() * dy.double()).sum())
        num, ana = (loss(1e-2) - loss(-1e-2)) / 2e-2, float((grad.double() * v.double()).sum())
        size = float((grad.double().square().sum() * v.double().square().sum()).sqrt())
        assert abs(num - ana) <= 1e-3 * size, (k, num, ana, size)


def test_many_rows_are_summed_in_a_fixed_order():
    gen = torch.Generator().manual_seed(2)
    x, dy = torch.randn(5000, 264, generator=gen).bfloat16().to(DEV), torch.randn(5000, 264, generator=gen).bfloat16().to(DEV)
    w = torch.rand(264, generator=gen).to(DEV)
    _, mean, rstd = ssd.norm_fwd(x, w, want_stats=True)
    a, b = ssd.norm_bwd(dy, x, w, mean, rstd), ssd.norm_bwd(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    hat = (R.up(x) - R.up(mean)[:, None]) * R.up(rstd)[:, None]
    R.check(a.dweight, (R.up(dy) * hat).sum(0), torch.float32, TOL_SUM, "dweight")
    R.check(a.dbias, R.up(dy).sum(0), torch.float32, TOL_SUM, "dbias")
