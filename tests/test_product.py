"""The matrix product with its epilogue (linear_fwd, linear_bwd) and the gated product (gated_fwd,
gated_bwd) against float64, within bounds that follow their roundings value by value
(ffn_ref)."""
import pytest
import torch

import ffn_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

SHAPES = [  # rows, inner, outer
    (1, 1, 1), (1, 8, 16), (2, 7, 3), (1, 2048, 520), (3, 1000, 264), (5, 64, 64), (16, 256, 96), (17, 129, 33),
    (31, 72, 200), (32, 300, 4300), (9, 136, 4104), (45, 200, 4100), (64, 72, 4200), (48, 512, 352), (40, 1100, 4000), (64, 264, 136), (65, 72, 136), (128, 64, 128), (129, 128, 127), (130, 200, 264),
    (255, 777, 129), (300, 96, 520), (513, 640, 392), (700, 72, 1032), (1030, 136, 520),
]
# enough tiles for the large ones, in each of the products: forward, by x, by the weight
LARGE = [(2901, 200, 2840), (2901, 2840, 72), (72, 2840, 2904)]
# large enough to have unaligned operands laid out anew first
UNALIGNED = [(1500, 1001, 1203), (1203, 777, 2050), (900, 2001, 1600)]
LARGE_GATED = [(2901, 200, 1424), (2901, 2840, 40), (72, 2840, 1456)]
DTYPES = [torch.float32, torch.bfloat16]


def make(m, k, n, dtype, seed, bias=True, residual=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype)
    return (r(m, k), r(n, k, std=k ** -0.5), r(n, std=0.3) if bias else None, r(m, n) if residual else None, r(m, n))


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_linear(shape, dtype, act):
    m, k, n = shape
    full = act is not None
    x, w, b, r, dy = make(m, k, n, dtype, m + k + n, bias=full, residual=act != "gelu")
    X, W, B, Rs, G = dev(x, w, b, r, dy)
    y, pre = ssd.linear_fwd(X, W, B, Rs, act=act, keep=True)
    assert (pre is None) == (act is None)
    y2 = ssd.linear_fwd(X, W, B, Rs, act=act)
    g = ssd.linear_bwd(G, X, W, B, pre, act=act)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    R.check_linear(dtype, (y, pre) + g, x, w, b, r, act, dy)


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_linear_in_large_tiles(shape):
    test_linear(shape, torch.bfloat16, "silu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", UNALIGNED, ids=str)
def test_unaligned_and_long(shape, dtype):
    test_linear(shape, dtype, "silu")
    test_linear(shape, dtype, None)
    test_gated(shape, dtype, "gelu")


@pytest.mark.parametrize("shape", [(4095, 777, 2051), (2561, 2047, 2051)], ids=str)
def test_laid_out_with_an_odd_last_value(shape):
    """bfloat16 operands that are laid out anew (in a workspace that holds both) and whose lines end
    with half of 4 bytes."""
    m, k, n = shape
    dims = ssd.ProductDims(m, k, n, ssd._DTYPE_CODE[torch.bfloat16], 0, k, n, n)
    assert ssd.lib().ssd_linear_fwd_workspace_bytes(dims) >= 2 * (m + n) * k
    test_linear(shape, torch.bfloat16, "silu")


@pytest.mark.parametrize("shape", LARGE_GATED, ids=str)
def test_gated_in_large_tiles(shape):
    test_gated(shape, torch.bfloat16, "silu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(shape, dtype, act):
    m, k, f = shape
    x, w, b, _, _ = make(m, k, 2 * f, dtype, m + 3 * k + f, bias=act == "silu", residual=False)
    dh = make(m, 1, f, dtype, 5)[4]
    X, W, B, G = dev(x, w, b, dh)
    h, pre = ssd.gated_fwd(X, W, B, act=act, keep=True)
    h2 = ssd.gated_fwd(X, W, B, act=act)
    g = ssd.gated_bwd(G, X, W, B, pre, act=act)
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    R.check_gated(dtype, (h, pre) + g, x, w, b, act, dh)


VIEWS = {  # name: (elements between rows beyond the row, elements before the first)
    "rows apart": (24, 0), "rows off 16 bytes": (3, 0), "start off 16 bytes": (8, 1), "half of wider rows": (1040, 520),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("shape", [(9, 64, 72), (200, 520, 264), (150, 131, 70)], ids=str)
def test_views(shape, dtype, view):
    """x, residual and dy as views of larger buffers whose other elements are NaN."""
    m, k, n = shape
    apart, before = VIEWS[view]
    x, w, b, r, dy = make(m, k, n, dtype, 1)

    def inside(t):
        buf = torch.full((before + t.shape[0] * (t.shape[1] + apart),), float("nan"), dtype=dtype)
        v = torch.as_strided(buf, t.shape, (t.shape[1] + apart, 1), before)
        v.copy_(t)
        return torch.as_strided(buf.to(DEV), t.shape, (t.shape[1] + apart, 1), before)
    X, Rs, G = inside(x), inside(r), inside(dy)
    W, B = dev(w, b)
    y, pre = ssd.linear_fwd(X, W, B, Rs, act="silu", keep=True)
    g = ssd.linear_bwd(G, X, W, B, pre, act="silu")
    R.check_linear(dtype, (y, pre) + g, x, w, b, r, "silu", dy)
    y = ssd.linear_fwd(X, W, B, Rs)
    g = ssd.linear_bwd(G, X, W, B)
    R.check_linear(dtype, (y, None) + g, x, w, b, r, None, dy)
    w2 = make(m, k, 2 * n, dtype, 2)[1]
    h, pre = ssd.gated_fwd(X, w2.to(DEV), keep=True)
    g = ssd.gated_bwd(G, X, w2.to(DEV), None, pre)
    R.check_gated(dtype, (h, pre) + g, x, w2, None, "silu", dy)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_row_for_all(dtype):
    """Rows of stride 0: x, residual and dy one row broadcast."""
    m, k, n = 70, 136, 200
    x, w, b, r, dy = (t[:1].expand(m, -1) if i in (0, 3, 4) else t for i, t in enumerate(make(m, k, n, dtype, 3)))
    one = lambda t: t[:1].contiguous().to(DEV).expand(m, -1)
    W, B = dev(w, b)
    y = ssd.linear_fwd(one(x), W, B, one(r))
    g = ssd.linear_bwd(one(dy), one(x), W, B)
    R.check_linear(dtype, (y, None) + g, x, w, b, r, None, dy)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(40, 72, 136), (300, 520, 264)], ids=str)
def test_needed_gradients_alone(shape, dtype):
    m, k, n = shape
    x, w, b, _, dy = make(m, k, n, dtype, 4)
    X, W, B, G = dev(x, w, b, dy)
    _, pre = ssd.linear_fwd(X, W, B, act="gelu", keep=True)
    whole = ssd.linear_bwd(G, X, W, B, pre, act="gelu")
    for i in range(3):
        need = [j == i for j in range(3)]
        g = ssd.linear_bwd(G, X, W, B, pre, act="gelu", need=need)
        for j in range(3):
            assert torch.equal(g[j], whole[j]) if j == i else g[j] is None
    assert ssd.linear_bwd(G, X, W, None, pre, act="gelu", need=(False, False, True)) == (None, None, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_not_finite_stays_in_its_row(dtype):
    """An infinity or NaN in a row of x reaches that row of the results alone; values beside a
    partial tile never count."""
    m, k, n = 37, 200, 136
    x, w, b, r, _ = make(m, k, n, dtype, 6)
    X, W, B, Rs = dev(x, w, b, r)
    clean = ssd.linear_fwd(X, W, B, Rs, act="silu")
    h = ssd.gated_fwd(X, W, B)
    X2 = X.clone()
    X2[5, 3], X2[36, 199] = float("inf"), float("nan")
    rows = torch.ones(m, dtype=torch.bool)
    rows[[5, 36]] = False
    assert torch.equal(ssd.linear_fwd(X2, W, B, Rs, act="silu")[rows], clean[rows])
    got = ssd.gated_fwd(X2, W, B)
    assert torch.equal(got[rows], h[rows])
    assert not torch.isfinite(got[36]).any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_far_from_zero(act):
    """The activations and their derivatives over the range in which they are not 0 or the
    identity, by a product with the identity."""
    v = torch.cat([torch.linspace(-14, 14, 4001), torch.tensor([-1e30, -200.0, 0.0, 200.0, 1e30])])[:, None].contiguous()
    one = torch.ones(1, 1)
    X, W = dev(v, one)
    y, pre = ssd.linear_fwd(X, W, act=act, keep=True)
    g = ssd.linear_bwd(torch.ones_like(X), X, W, None, pre, act=act, need=(True, False, False))
    ref, dref = R.act(R.up(v), act), R.dact(R.up(v), act)
    ref[-5:] = torch.tensor([0.0, 0.0, 0.0, 200.0, 1e30])[:, None]
    dref[-5:] = torch.tensor([0.0, 0.0, 0.5, 1.0, 1.0])[:, None]
    R.inside(y, ref, R.ACT * ref.abs() + 1e-30, act)
    R.inside(g.dx, dref, torch.full_like(dref, R.ACT), "its derivative")


def test_calls_repeat_bit_for_bit():
    for m, k, n in ((1, 2048, 1024), (48, 2048, 704), (600, 1024, 264)):
        x, w, b, r, dy = dev(*make(m, k, n, torch.bfloat16, 9))
        a = ssd.linear_fwd(x, w, b, r), *ssd.linear_bwd(dy, x, w, b)
        for _ in range(3):
            c = ssd.linear_fwd(x, w, b, r), *ssd.linear_bwd(dy, x, w, b)
            assert all(torch.equal(p, q) for p, q in zip(a, c))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(256, 256, 256), (640, 333, 517), (1024, 520, 264), (77, 1000, 1040), (900, 70, 1999)], ids=str)
def test_both_gradients_are_those_of_each_alone(shape, dtype):
    """Whether one launch takes both products or one each; with dy and x off 16 bytes too."""
    m, k, n = shape
    x, w, b, _, dy = make(m, k, n, dtype, 6)
    X, W, B, G = dev(x, w, b, dy)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    for xs, gs in ((X, G), (off(X), G), (X, off(G))):
        both = ssd.linear_bwd(gs, xs, W, B)
        x_alone = ssd.linear_bwd(gs, xs, W, B, need=(True, False, False)).dx
        w_alone = ssd.linear_bwd(gs, xs, W, B, need=(False, True, False)).dweight
        y = ssd.linear_fwd(xs, W, B)
        R.check_linear(dtype, (y, None) + both, x, w, b, None, None, dy)
        R.check_linear(dtype, (y, None, x_alone, w_alone, both.dbias), x, w, b, None, None, dy)
