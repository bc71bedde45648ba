"""The norms around a residual at infinite parameters and gates, and at many narrow rows."""
import pytest
import torch

from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16]
INF = float("inf")
EPS = 1e-5
# a whole number of 16 bytes, rows that end inside an access, and rows that registers do not hold
CHANNELS = [1024, 1025, 1029, 333, 8201]


def shared(d, dtype):
    """The last channel that a row's last access shares with the one before it, if any are."""
    v = 16 // torch.empty((), dtype=dtype).element_size()
    return d - 1 - d % v


def rand(d, dtype, n, rows=5):
    gen = torch.Generator().manual_seed(d)
    return [(torch.randn(rows, d, generator=gen).to(dtype)).to(DEV) for _ in range(n)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", CHANNELS)
@pytest.mark.parametrize("which", ["post", "scale"])
def test_an_infinite_parameter_stays_in_its_channel(which, d, dtype):
    """The sum of squares of the total is infinite and not NaN: the normed row is 0 but for the
    infinite channel itself."""
    branch, residual = rand(d, dtype, 2)
    at = shared(d, dtype)
    par = torch.ones(d, device=DEV)
    par[at] = INF
    post, scale = (par, None) if which == "post" else (None, par)
    y, total = ssd.residual_norm_fwd(branch, residual, None, post, scale, torch.ones(d, device=DEV))
    others = [c for c in range(d) if c != at]
    assert total[:, at].isinf().all() and total[:, others].isfinite().all()
    assert (y[:, others] == 0).all() and y[:, at].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", CHANNELS)
def test_an_infinite_weight_in_the_gradient(d, dtype):
    """Without the second norm: h = dtotal post is infinite in one channel, so is the mean of h that,
    and so every gradient of the row: infinite by the formula, NaN in the channel alone
    (infinity - infinity) or infinite there too."""
    branch, dtotal = rand(d, dtype, 2)
    at = shared(d, dtype)
    post = torch.ones(d, device=DEV)
    post[at] = INF
    _, _, stats = ssd.residual_norm_fwd(branch, None, None, post, want_stats=True)
    g = ssd.residual_norm_bwd(None, dtotal, branch, None, None, post, None, None, stats)
    others = [c for c in range(d) if c != at]
    assert g.dbranch[:, others].isinf().all()
    assert g.dpost_weight[others].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", CHANNELS + [3])
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinite_gate_in_the_gradient(sign, d, dtype):
    """silu is v at +infinity with a derivative of 1, and 0 at -infinity with a derivative of 0:
    dgate = dtotal scale branch, or 0."""
    branch, residual, gate, dtotal = rand(d, dtype, 4)
    branch = branch.abs() + 1
    dtotal = dtotal.abs() + 1
    at = shared(d, dtype) if d > 8 else 1
    gate[:, at] = sign * INF
    scale = torch.full((d,), 0.5, device=DEV)
    others = [c for c in range(d) if c != at]
    _, total, stats = ssd.residual_norm_fwd(branch, residual, gate, None, scale, want_stats=True)
    g = ssd.residual_norm_bwd(None, dtotal, branch, residual, gate, None, scale, None, stats)
    assert total[:, others].isfinite().all() and g.dbranch[:, others].isfinite().all()
    if sign > 0:
        assert (total[:, at] == INF).all() and (g.dbranch[:, at] == INF).all()
        want = (dtotal[:, at].float() * 0.5 * branch[:, at].float()).to(dtype)
    else:
        assert torch.equal(total[:, at], residual[:, at]) and (g.dbranch[:, at] == 0).all()
        want = torch.zeros_like(g.dgate[:, at])
        assert g.dscale[at] == 0
    assert torch.equal(g.dgate[:, at], want) and g.dgate[:, others].isfinite().all()


@pytest.mark.parametrize("dtype,d", [(torch.float32, 4), (torch.float32, 7), (torch.float32, 3), (torch.bfloat16, 3),
                                     (torch.bfloat16, 8)], ids=str)
def test_many_narrow_rows(dtype, d):
    """More rows than a launch has workgroups of 1024 threads.  Float32 sums of a row have at most 7
    terms: 4e-5 of the largest value as for other rows, and half a step of what is stored; a column's sum
    is rows / 512 terms in turn, then 512: that many times 2^-24 of the terms' sizes, and 4e-5 of
    them for the terms themselves."""
    rows = 4_200_001
    gen = torch.Generator(device=DEV).manual_seed(d)
    act = lambda: torch.randn(rows, d, generator=gen, device=DEV).to(dtype)
    par = lambda: 1 + 0.3 * torch.randn(d, generator=gen, device=DEV)
    branch, residual, dy, dtotal, post, scale, pre = act(), act(), act(), act(), par(), par(), par()
    branch.add_(torch.where(branch < 0, -1., 1.).to(dtype))       # no row of a norm near 0, whose inverse is large
    residual.mul_(0.25)
    y, total, stats = ssd.residual_norm_fwd(branch, residual, None, post, scale, pre, EPS, want_stats=True)
    g = ssd.residual_norm_bwd(dy, dtotal, branch, residual, None, post, scale, pre, stats)
    torch.cuda.synchronize()
    B, R, P, S, Q = (t.double().requires_grad_(True) for t in (branch, residual, post, scale, pre))
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    tr = R + rms(B) * P * S
    yr = rms(tr) * Q
    grads = torch.autograd.grad((yr, tr), (B, R, P, S, Q), (dy.double(), dtotal.double()))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    with torch.no_grad():
        inv = 1 / torch.sqrt((tr * tr).mean(1, keepdim=True) + EPS)
        ds = dtotal.double().abs() + 2 * inv * (dy.double() * Q).abs()
        dt = 2 * ds * (S * P).abs() / torch.sqrt((B * B).mean(1, keepdim=True) + EPS)
        near = lambda got, ref, size: ((got.double() - ref).abs() <= 4e-5 * size + half * ref.abs()).all()
        assert near(total, tr, tr.abs().max()) and near(y, yr, yr.abs().max())
        assert near(g.dresidual, grads[1], ds.max(1, keepdim=True).values) and near(g.dbranch, grads[0], dt.max(1, keepdim=True).values)
        count = 2.0 ** -24 * (rows / 512 + 512) + 4e-5
        that = rms(B)
        for got, ref, terms in ((g.dpost_weight, grads[2], ds * (S * that).abs()), (g.dscale, grads[3], ds * (that * P).abs()),
                                (g.dpre_weight, grads[4], (dy.double() * rms(tr)).abs())):
            assert ((got.double() - ref).abs() <= count * terms.sum(0)).all()
