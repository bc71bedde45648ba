"""Offsets beyond 2^31 elements and strides beyond 2^31 bytes, against the same values computed a
few rows at a time."""
import pytest
import torch

import ffn_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROWS, WIDE = 70001, 32768                  # 2.29e9 elements


def close(got, ref, tol=2.0 ** -6):
    """bfloat16 results of float32 references: half a step and twice that for what entered them."""
    err = (got.float() - ref).abs().max()
    assert float(err) <= tol * float(ref.abs().max()), (float(err), float(ref.abs().max()))


@pytest.fixture(scope="module")
def x():
    gen = torch.Generator(device=DEV).manual_seed(1)
    t = torch.empty(ROWS, WIDE, device=DEV, dtype=torch.bfloat16)
    for i in range(0, ROWS, 8192):
        t[i:i + 8192] = torch.randn(min(8192, ROWS - i), WIDE, generator=gen, device=DEV)
    return t


PICK = [0, 1, 65535, 65536, 65537, 70000]


def test_products(x):
    gen = torch.Generator(device=DEV).manual_seed(2)
    w = (torch.randn(96, WIDE, generator=gen, device=DEV) * WIDE ** -0.5).bfloat16()
    y = ssd.linear_fwd(x, w)
    close(y[PICK], x[PICK].float() @ w.float().t())
    h, pre = ssd.gated_fwd(x, w, keep=True)
    g, u = (x[PICK].float() @ w.float().t()).chunk(2, 1)
    close(h[PICK], torch.nn.functional.silu(g) * u)
    dy = torch.randn(ROWS, 96, generator=gen, device=DEV).bfloat16()
    got = ssd.linear_bwd(dy, x, w, need=(True, True, False))
    close(got.dx[PICK], dy[PICK].float() @ w.float())
    cols = [0, 1, 32767]
    close(got.dweight[:, cols], dy.float().t() @ x[:, cols].float())
    dh = dy[:, :48]
    got = ssd.gated_bwd(dh, x, w, None, pre, need=(True, False, False))
    d = torch.cat([dh[PICK].float() * u * R.dact(g, "silu"), dh[PICK].float() * torch.nn.functional.silu(g)], 1)
    close(got.dx[PICK], d @ w.float(), 2.0 ** -5)


def test_residual_norm(x):
    for width in (WIDE, 8192):                      # wider than registers, and not
        t = x.view(-1, width)
        one = torch.ones(width, device=DEV)
        rows = [0, 1, t.shape[0] // 2, t.shape[0] - 1]
        y, total, stats = ssd.residual_norm_fwd(t, t, None, one, one, one, want_stats=True)
        b = t[rows].float()
        s = b + b / torch.sqrt((b * b).mean(1, keepdim=True) + 1e-5)
        close(total[rows], s)
        close(y[rows], s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-5))
        g = ssd.residual_norm_bwd(None, t, t, None, None, None, one, None, stats)
        assert torch.equal(g.dbranch[rows], t[rows])
        del y, total, g


def test_clip(x):
    flat = x.view(-1)
    out = torch.empty_like(flat)
    n = ssd.clip_grads([flat], 1.0, out=[out])
    ref = float(torch.sqrt(sum(p.double().square().sum() for p in flat.split(1 << 28))))
    assert abs(float(n) - ref) <= 2.0 ** -22 * ref
    at = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, flat.numel() - 1], device=DEV)
    close(out[at], flat[at].float() / ref)


@pytest.mark.parametrize("start", [0, 1])
def test_strides_beyond_two_gigabytes_a_tile(start):
    """Rows 5e6 elements apart, on and off 16 bytes: a tile's rows span more than 32 bits hold."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    m, k, n, apart = 300, 200, 72, 5000000
    buf = torch.empty(start + m * apart, device=DEV, dtype=torch.bfloat16)
    x = torch.as_strided(buf, (m, k), (apart, 1), start)
    x.copy_(torch.randn(m, k, generator=gen, device=DEV))
    w, dy = torch.randn(n, k, generator=gen, device=DEV).bfloat16(), torch.randn(m, n, generator=gen, device=DEV).bfloat16()
    c = x.contiguous()
    close(ssd.linear_fwd(x, w), c.float() @ w.float().t())
    close(ssd.linear_bwd(dy, x, w).dweight, dy.float().t() @ c.float())
    close(ssd.linear_fwd(x[:20], w), c[:20].float() @ w.float().t())
    y, total = ssd.residual_norm_fwd(x, x, x, pre_weight=torch.ones(k, device=DEV))
    y2, total2 = ssd.residual_norm_fwd(c, c, c, pre_weight=torch.ones(k, device=DEV))
    assert float((y.float() - y2.float()).abs().max()) <= 2.0 ** -7 * float(y2.float().abs().max())
    assert float((total.float() - total2.float()).abs().max()) <= 2.0 ** -7 * float(total2.float().abs().max())
