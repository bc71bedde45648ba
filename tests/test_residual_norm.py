"""The norms around a residual (residual_norm_fwd, residual_norm_bwd) against float64.

Tolerance: the means of squares are sums of D float32 terms in runs of at most 32 a lane and a
tree across lanes: 40 * 2^-24 of the terms' sizes, and each of the two norms' sums enters every
later value: 4e-5 of the largest value for values of a row (twice the layer norm's bound, for two
norms), 1e-4 for sums over rows, as the layer norm's.  Where terms cancel in every element their
size counts."""
import itertools

import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL, TOL_SUM = 4e-5, 1e-4
EPS = 1e-5


def rms(v):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def reference(branch, residual, gate, post, scale, pre):
    t = branch if gate is None else branch * gate * torch.sigmoid(gate)
    p = t if post is None else rms(t) * post
    s = p if scale is None else p * scale
    total = s if residual is None else residual + s
    return (None if pre is None else rms(total) * pre), total


def make(rows, D, dtype, given, seed=0, extra=0):
    """branch, residual, gate (views with `extra` elements between rows), post, scale, pre, dy,
    dtotal; `given`: which of residual, gate, post, scale, pre."""
    gen = torch.Generator().manual_seed(seed + rows + D)
    act = lambda std=1.0: (torch.randn(rows, D + extra, generator=gen) * std).to(dtype)[:, :D]
    par = lambda at: at + 0.3 * torch.randn(D, generator=gen)
    t = [act(), act(2.0), act(1.5), par(1.0), par(0.7), par(1.0), act(), act()]
    for i, on in enumerate(given):
        if not on:
            t[1 + i] = None
    if not given[4]:
        t[6] = None
    return t


def to_dev(t):
    """On the device with the same strides."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.to(DEV)
    full = torch.empty(t.stride(0) * t.shape[0], dtype=t.dtype, device=DEV)
    v = torch.as_strided(full, t.shape, t.stride())
    v.copy_(t)
    return v


def check_all(tensors, dtype, got, tol=TOL, tol_sum=TOL_SUM):
    y, total, g = got
    leaves = [R.up(t) for t in tensors]
    names = ["branch", "residual", "gate", "post_weight", "scale", "pre_weight"]
    for t in leaves[:6]:
        if t is not None:
            t.requires_grad_(True)
    yr, tr = reference(*leaves[:6])
    R.check(total, tr, dtype, tol, "total")
    assert (y is None) == (yr is None)
    if y is not None:
        R.check(y, yr, dtype, tol, "y")
    if g is None:
        return
    on = [i for i in range(6) if leaves[i] is not None]
    grads = R.grads((yr, tr) if yr is not None else (tr,), (leaves[6], leaves[7]) if yr is not None else (leaves[7],),
                    [leaves[i] for i in on])
    order = [g.dbranch, g.dresidual, g.dgate, g.dpost_weight, g.dscale, g.dpre_weight]
    # the sizes of the terms that a gradient is a difference of
    ds = torch.zeros(1, dtype=R.F64) if leaves[7] is None else leaves[7].abs()
    if leaves[6] is not None:
        inv = 1.0 / torch.sqrt((tr.detach() ** 2).mean(1, keepdim=True) + EPS)
        ds = ds + 2 * inv * (leaves[6] * leaves[5].detach()).abs()
    dt = ds * (1 if leaves[4] is None else leaves[4].detach().abs())
    b, z = leaves[0].detach(), None if leaves[2] is None else leaves[2].detach()
    t = b if z is None else b * z * torch.sigmoid(z)
    if leaves[3] is not None:
        dt = 2 * dt * leaves[3].detach().abs() / torch.sqrt((t ** 2).mean(1, keepdim=True) + EPS)
    scales = {0: float(dt.max()), 1: float(ds.max()), 2: float((dt * b.abs()).max()) if z is not None else 0.0}
    for i, ref in zip(on, grads):
        what = "gradient of " + names[i]
        if i < 3:
            R.check(order[i], ref, dtype, tol, what, scale=scales[i])
        else:
            R.check(order[i], ref, torch.float32, tol_sum, what, scale=float(ds.max()))
    assert all((order[i] is None) == (leaves[i] is None) for i in range(6))


def same(a, b):
    return torch.equal(a.nan_to_num(1e4), b.nan_to_num(1e4))


def run(t):
    d = [to_dev(v) for v in t]
    y, total, stats = ssd.residual_norm_fwd(*d[:6], EPS, want_stats=True)
    y2, total2 = ssd.residual_norm_fwd(*d[:6], EPS)
    g = ssd.residual_norm_bwd(d[6], d[7], *d[:6], stats)
    torch.cuda.synchronize()
    assert same(total, total2) and (y is None or same(y, y2))
    return y, total, g


SHAPES = [  # rows, D, elements between rows beyond D
    (1, 1, 0), (1, 768, 0), (3, 2, 0), (2, 63, 1), (5, 64, 0), (4, 65, 3), (7, 255, 0), (6, 257, 0), (9, 512, 8),
    (3, 520, 0), (700, 1024, 0), (11, 1025, 0), (5, 2048, 2048), (3, 2056, 0), (2, 4095, 0), (4, 4096, 0), (3, 4104, 8),
    (3, 8192, 0), (3, 5001, 1), (2, 8190, 3), (600, 1001, 0), (2, 8199, 0), (3, 16384, 0), (1500, 40, 0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_everything_given(shape, dtype):
    rows, D, extra = shape
    t = make(rows, D, dtype, [True] * 5, extra=extra)
    check_all(t, dtype, run(t))


@pytest.mark.parametrize("given", list(itertools.product([False, True], repeat=5)), ids=str)
@pytest.mark.parametrize("D", [200, 4100, 8201])
def test_each_combination(given, D):
    """residual, gate, post_weight, scale and pre_weight given or not, in registers and not."""
    t = make(5, D, torch.bfloat16, given, seed=3)
    check_all(t, torch.bfloat16, run(t))
    if given[4]:                       # without a gradient of total
        t[7] = None
        check_all(t, torch.bfloat16, run(t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [96, 1000, 8201])
def test_total_in_place_of_residual(dtype, D):
    t = make(9, D, dtype, [True] * 5, seed=5)
    d = [v.to(DEV) for v in t]
    y, total = ssd.residual_norm_fwd(*d[:6], EPS)
    before = d[1]._version
    y2, total2 = ssd.residual_norm_fwd(*d[:6], EPS, total=d[1])
    assert total2 is d[1] and d[1]._version > before
    assert torch.equal(y, y2) and torch.equal(total, total2)


def test_rows_of_zeros():
    """A row of zeros stays zeros, and its gradients are finite."""
    t = make(6, 300, torch.float32, [True] * 5, seed=7)
    t[0][2] = 0.0
    t[1][2] = 0.0
    t[2][4] = 0.0
    y, total, g = run(t)
    assert float(y[2].abs().max()) == 0.0 and float(total[2].abs().max()) == 0.0
    assert all(torch.isfinite(v).all() for v in g)


def test_what_is_not_finite_stays_in_its_row():
    t = make(8, 520, torch.bfloat16, [True] * 5, seed=8)
    y, total, g = run(t)
    t[0][3, 5], t[1][6, 519] = float("nan"), float("inf")
    y2, total2, g2 = run(t)
    rows = [0, 1, 2, 4, 5, 7]
    for a, b in ((y, y2), (total, total2), (g.dbranch, g2.dbranch), (g.dgate, g2.dgate), (g.dresidual, g2.dresidual)):
        assert torch.equal(a[rows], b[rows])


def test_gradient_against_differences():
    """Central differences with a step of 1e-2: truncation (1e-2)^2 times third derivatives of a
    few units, and rounding 1e-6 / 1e-2, stay below 2e-3."""
    gen = torch.Generator().manual_seed(1)
    t = [v.to(DEV) for v in make(6, 300, torch.float32, [True] * 5, seed=9)]
    _, _, stats = ssd.residual_norm_fwd(*t[:6], EPS, want_stats=True)
    g = ssd.residual_norm_bwd(t[6], t[7], *t[:6], stats)
    for k, grad in enumerate(g):
        v = torch.randn(t[k].shape, generator=gen).to(DEV)

        def loss(s):
            e = list(t[:6])
            e[k] = t[k] + s * v
            y, total = ssd.residual_norm_fwd(*e, EPS)
            return float((y.double() * t[6].double()).sum() + (total.double() * t[7].double()).sum())
        num, ana = (loss(1e-2) - loss(-1e-2)) / 2e-2, float((grad.double() * v.double()).sum())
        size = float((grad.double().square().sum() * v.double().square().sum()).sqrt())
        assert abs(num - ana) <= 2e-3 * size, (k, num, ana, size)


def test_many_rows_are_summed_in_a_fixed_order():
    t = [v.to(DEV) for v in make(5000, 264, torch.bfloat16, [True] * 5, seed=10)]
    _, _, stats = ssd.residual_norm_fwd(*t[:6], EPS, want_stats=True)
    a, b = (ssd.residual_norm_bwd(t[6], t[7], *t[:6], stats) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [1024, 1025, 1029, 333])
def test_an_infinite_gate_stays_in_its_channel(d, dtype):
    """Channels that a row's last access shares with the one before it are read twice and count
    once, whatever they hold: the sum of squares is infinite and not NaN, so the normed row is
    0 and the total the residual, but for the infinite channel itself."""
    rows = 5
    gen = torch.Generator().manual_seed(d)
    branch, residual, gate = (torch.randn(rows, d, generator=gen).to(dtype) for _ in range(3))
    at = d - 3
    branch[:, at] = 1.
    gate[:, at] = float("inf")
    ones = torch.ones(d, device=DEV)
    y, total = ssd.residual_norm_fwd(branch.to(DEV), residual.to(DEV), gate.to(DEV), ones)
    assert y is None
    others = [c for c in range(d) if c != at]
    assert torch.equal(total.cpu()[:, others], residual[:, others]) and total[:, at].isnan().all()
    y, total = ssd.residual_norm_fwd(branch.to(DEV), residual.to(DEV), gate.to(DEV), None, None, ones)
    assert total[:, at].isinf().all() and total[:, others].isfinite().all()
    assert (y[:, others] == 0).all() and y[:, at].isnan().all()
