"""The products where they are cut, joined and laid out in each of their ways: the same bits at every
call, and what is not finite.

A row of x (or of dy) is a row of the result, so nothing of one row may reach another: not by the
rows that a tile repeats past the last one, nor by the values beside a row's last ones, nor by
zeros past K.  Results of clean rows have to be the same bits with and without it."""
import pytest
import torch

import ffn_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16]
INF, NAN = float("inf"), float("nan")

# rows, inner, outer, and what the forward's workspace shows of its path: more than nothing where K is
# split, both operands where they are laid out anew, less than that where they pass through registers
PATHS = {
    "direct, K ends in a step": (130, 200, 264, None),
    "through registers": (150, 131, 70, "registers"),
    "K split and joined": (100, 4096, 64, "split"),
    "laid out anew": (2561, 2047, 2051, "laid out"),
    "tiles of 256": (2901, 200, 2840, None),
}


def make(m, k, n, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(dtype)
    return r(m, k), r(n, k, std=k ** -0.5), r(n, std=0.3), r(m, n), r(m, n)


def check_path(m, k, n, dtype, path, gated):
    dims = ssd.ProductDims(m, k, n, ssd._DTYPE_CODE[dtype], 0, k, n, n)
    L = ssd.lib()
    got = (L.ssd_gated_fwd_workspace_bytes if gated else L.ssd_linear_fwd_workspace_bytes)(dims)
    both = (m + n * (2 if gated else 1)) * k * (2 if dtype == torch.bfloat16 else 4)
    if path == "split":
        assert got > 0
    elif path == "laid out":
        assert got >= both
    elif path == "registers":
        assert got < both


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_gated_calls_repeat_bit_for_bit(path, dtype):
    m, k, n, kind = PATHS[path]
    f = n // 2
    check_path(m, k, f, dtype, kind if kind != "registers" else None, True)
    x, w, b, _, _ = make(m, k, 2 * f, dtype, 1)
    dh = make(m, 1, f, dtype, 2)[4]
    first = None
    for _ in range(4):
        h, pre = ssd.gated_fwd(x, w, b, keep=True)
        got = (h, pre) + ssd.gated_bwd(dh, x, w, b, pre)
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(first, got))


def bad_rows(t):
    """The same with infinities of both signs in a row and a NaN at the end of the last one; the others."""
    m, k = t.shape
    t = t.clone()
    t[m // 2, 3], t[m // 2, k - 1], t[m - 1, k - 1] = INF, -INF, NAN
    rows = torch.ones(m, dtype=torch.bool, device=DEV)
    rows[[m // 2, m - 1]] = False
    return t, rows


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_a_row_stays_in_its_row_forward(path, dtype):
    m, k, n, kind = PATHS[path]
    x, w, b, r, _ = make(m, k, n, dtype, 1)
    check_path(m, k, n, dtype, kind, False)
    x2, rows = bad_rows(x)
    for act in (None, "silu"):
        clean, got = (ssd.linear_fwd(v, w, b, r, act=act) for v in (x, x2))
        assert torch.equal(got[rows], clean[rows])
        assert got[m - 1].isnan().all()
    f = n // 2
    check_path(m, k, f, dtype, None, True)
    clean, got = (ssd.gated_fwd(v, w[:2 * f], b[:2 * f]) for v in (x, x2))
    assert torch.equal(got[rows], clean[rows])
    assert got[m - 1].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("path", PATHS)
def test_a_row_stays_in_its_row_by_x(path, act, dtype):
    """dx: a row of dy is a row of dx; the sums run over the outer dimension."""
    m, n, k, _ = PATHS[path]                           # the path's K is what dx sums over
    x, w, b, _, dy = make(m, k, n, dtype, 2)
    _, pre = ssd.linear_fwd(x, w, b, act=act, keep=True)
    dy2, rows = bad_rows(dy)
    for need in ((True, False, False), (True, True, True)):
        clean, got = (ssd.linear_bwd(v, x, w, b, pre, act=act, need=need).dx for v in (dy, dy2))
        assert torch.equal(got[rows], clean[rows])
        assert got[m - 1].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("path", PATHS)
def test_a_column_stays_in_its_column_by_the_weight(path, act, dtype):
    """dweight sums over the rows: a column of dy is a row of it, a column of x a column."""
    n, m, k, _ = PATHS[path]                           # the path's K is the rows here
    x, w, b, _, dy = make(m, k, n, dtype, 3)
    _, pre = ssd.linear_fwd(x, w, b, act=act, keep=True)
    dyt, rows = bad_rows(dy.t().contiguous())
    xt, cols = bad_rows(x.t().contiguous())
    dy2, x2 = dyt.t().contiguous(), xt.t().contiguous()
    for need in ((False, True, False), (True, True, True)):
        clean = ssd.linear_bwd(dy, x, w, b, pre, act=act, need=need).dweight
        got = ssd.linear_bwd(dy2, x, w, b, pre, act=act, need=need).dweight
        assert torch.equal(got[rows], clean[rows]) and got[n - 1].isnan().all()
        got = ssd.linear_bwd(dy, x2, w, b, pre, act=act, need=need).dweight
        assert torch.equal(got[:, cols], clean[:, cols]) and got[:, k - 1].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_gated_row_stays_in_its_row_backward(dtype):
    for m, k, f in ((130, 200, 264), (150, 131, 35), (1500, 1001, 602)):
        x, w, b, _, _ = make(m, k, 2 * f, dtype, 4)
        dh = make(m, 1, f, dtype, 5)[4]
        _, pre = ssd.gated_fwd(x, w, b, keep=True)
        dh2, rows = bad_rows(dh)
        clean, got = (ssd.gated_bwd(v, x, w, b, pre).dx for v in (dh, dh2))
        assert torch.equal(got[rows], clean[rows]) and got[m - 1].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", ["outer", "inner"])
def test_one_row_by_many_columns(wide, dtype):
    """The weight's gradient of a single row, whose sums have one term: a line of k so long that a
    tile's offsets over further lines, which there are none of, pass 32 bits.  Zeros stand for them,
    whatever the row holds there."""
    n = 40_000_000
    # the value that line 54 (bfloat16) or 27 of a tile's first column wraps to
    at = 54 * n - 2 ** 31 if dtype == torch.bfloat16 else 27 * n - 2 ** 30
    assert 0 < at < n
    inner, outer = (8, n) if wide == "outer" else (n, 8)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1, inner, generator=gen, device=DEV).to(dtype)
    dy = torch.randn(1, outer, generator=gen, device=DEV).to(dtype)
    (dy if wide == "outer" else x)[0, at] = INF
    w = torch.zeros(outer, inner, dtype=dtype, device=DEV)
    got = ssd.linear_bwd(dy, x, w, need=(False, True, False)).dweight
    del w
    want = (dy.float().t() * x.float()).to(dtype)
    assert torch.equal(got, want)


def gated_with(m, k, f, dtype, keep, act="silu"):
    x, w, b, _, _ = make(m, k, 2 * f, dtype, 6)
    dh = make(m, 1, f, dtype, 7)[4]
    h, pre = ssd.gated_fwd(x, w, b, act=act, keep=keep)
    return (x, w, b, dh), (h, pre) + ssd.gated_bwd(dh, x, w, b, pre, act=act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_have_one_rounding_beside_their_own(act):
    """bfloat16, in the 2-norm: a gradient's terms are rounded once (the gradient by pre) and so is
    the result, two independent roundings of the same relative size, so sqrt 2 of what rounding the
    exact result leaves; with pre rounded too it is sqrt 3 and more.  The bias' gradient sums
    what is not rounded yet."""
    m, k, f = 2048, 1024, 1408
    (x, w, b, dh), got = gated_with(m, k, f, torch.bfloat16, True, act)
    assert got[1].dtype == torch.float32
    X, W, B = (t.double().requires_grad_(True) for t in (x, w, b))
    g, u = (X @ W.t() + B).chunk(2, 1)
    a = g * torch.sigmoid(g) if act == "silu" else g * torch.special.ndtr(g)
    ref = torch.autograd.grad(a * u, (X, W, B), dh.double())
    for name, mine, r, times in zip(("dx", "dweight", "dbias"), got[2:], ref, (1.55, 1.55, 1.05)):
        alone = (r.bfloat16().double() - r).norm()
        assert (mine.double() - r).norm() <= times * alone, name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 200, 72), (130, 200, 264), (150, 131, 35), (700, 1001, 602), (2901, 136, 1424)], ids=str)
def test_pre_in_either_type(shape, dtype):
    """float32 by keep=True, or x's own type: what is kept rounded is the same values rounded, and the
    gradients are off by no more than their roundings (value by value against float64)."""
    m, k, f = shape
    runs = [gated_with(m, k, f, dtype, keep) for keep in (True, torch.float32, dtype)]
    assert [r[1][1].dtype for r in runs] == [torch.float32, torch.float32, dtype]
    for p, q in zip(runs[0][1], runs[1][1]):
        assert torch.equal(p, q)
    assert torch.equal(runs[2][1][0], runs[0][1][0]) and torch.equal(runs[2][1][1], runs[0][1][1].to(dtype))
    for (x, w, b, dh), got in runs:
        R.check_gated(dtype, got, x, w, b, "silu", dh)
    n = 2 * f
    x, w, b, r, dy = make(m, k, n, dtype, 8)
    for keep in (True, dtype):
        y, pre = ssd.linear_fwd(x, w, b, r, act="gelu", keep=keep)
        assert pre.dtype == (torch.float32 if keep is True else dtype)
        R.check_linear(dtype, (y, pre) + ssd.linear_bwd(dy, x, w, b, pre, act="gelu"), x, w, b, r, "gelu", dy)
