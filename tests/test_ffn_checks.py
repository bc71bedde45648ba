"""What the operators of a layer's feed-forward half refuse (no GPU: every call fails before
anything is enqueued): the C ABI's status codes, the binding's tensor checks, and the versions
of tensors that a call writes."""
import ctypes

import pytest
import torch

from chunked_linear_recurrence_amd import ssd

F = 1 << 40                        # an aligned address that is never dereferenced
P = [F + (k << 36) for k in range(32)]


def lib():
    try:
        return ssd.lib()
    except RuntimeError:
        pytest.skip("libssdscan.so not built")


# ------------------------------------------------------------------------------- C ABI
def dims(m=40, k=32, n=16, dtype=0, reserved=0, xs=None, rs=None, gs=None):
    return ssd.ProductDims(m, k, n, dtype, reserved, k if xs is None else xs, n if rs is None else rs, n if gs is None else gs)


def linear_fwd(d, x=P[0], w=P[1], b=P[2], r=P[3], y=P[4], pre=P[5], flags=8, ws=P[6], n=1 << 32):
    return lib().ssd_linear_fwd(d, x, w, b, r, y, pre, flags, ws, n, None)


def gated_fwd(d, x=P[0], w=P[1], b=P[2], h=P[4], pre=P[5], flags=8, ws=P[6], n=1 << 32):
    return lib().ssd_gated_fwd(d, x, w, b, h, pre, flags, ws, n, None)


@pytest.mark.parametrize("fwd", [linear_fwd, gated_fwd])
def test_product_fwd_refusals(fwd):
    assert fwd(None) == 1
    assert fwd(dims(dtype=2)) == 3
    for bad in (dict(m=0), dict(k=0), dict(n=0), dict(m=-1), dict(reserved=1), dict(xs=-1)):
        assert fwd(dims(**bad)) == 2, bad
    for bad in (dict(m=1 << 31), dict(k=1 << 30), dict(n=1 << 30)):
        assert fwd(dims(**bad)) == 4, bad
    for bad in (dict(x=None), dict(w=None)):
        assert fwd(dims(), **bad) == 1, bad
    for flags in (1, 16, 8 | 32, 64):
        assert fwd(dims(), flags=flags) == 2, flags
    for bad in (dict(x=P[0] + 2), dict(w=P[1] + 1), dict(b=P[2] + 3), dict(pre=P[5] + 2)):
        assert fwd(dims(), **bad) == 5, bad
    assert fwd(dims(dtype=1), x=P[0] + 1) == 5
    for bad in (dict(pre=P[0] + 64), dict(pre=P[1]), dict(pre=P[4] + 8), dict(pre=P[2])):
        assert fwd(dims(), **bad) == 8, bad
    assert lib().ssd_last_error_message().decode() != ""
    # more tiles than a launch holds
    assert fwd(dims(m=1 << 22, k=1, n=1 << 21)) == 4


def test_linear_and_gated_refusals_of_their_own():
    assert linear_fwd(dims(), y=None) == 1 and gated_fwd(dims(), h=None) == 1
    assert linear_fwd(dims(rs=-3)) == 2 and linear_fwd(dims(), r=P[3] + 2) == 5
    assert linear_fwd(dims(), y=P[3]) == 8                          # not in place of the residual
    assert gated_fwd(dims(), flags=0) == 2                          # an activation is needed
    # strides of what is not given, and over one row, are not looked at
    assert linear_fwd(dims(rs=-3), r=None, y=P[0]) == 8
    assert linear_fwd(dims(m=1, xs=-1, rs=-1), y=P[0]) == 8


def test_workspaces():
    L = lib()
    assert L.ssd_linear_fwd_workspace_bytes(dims(m=0)) == 0 and L.ssd_gated_fwd_workspace_bytes(dims(dtype=5)) == 0
    for m in (1, 32):
        assert L.ssd_linear_fwd_workspace_bytes(dims(m, 4097, 4099, 1)) == 0
        assert L.ssd_gated_fwd_workspace_bytes(dims(m, 4097, 4099, 1)) == 0
    for fwd, size in ((linear_fwd, L.ssd_linear_fwd_workspace_bytes), (gated_fwd, L.ssd_gated_fwd_workspace_bytes)):
        d = dims(100, 8192, 64, 1)                                  # few tiles, many steps: K is cut
        need = size(d)
        assert need > 0
        assert fwd(d, n=need - 1) == 6 and fwd(d, ws=None) == 6
        assert fwd(d, ws=P[6] + 8, n=need) == 5 and fwd(d, ws=P[0], n=need) == 8
    d = dims(4095, 4095, 4095, 1)                                   # operands are laid out anew
    assert L.ssd_linear_fwd_workspace_bytes(d) >= 2 * 4095 * 4096 * 2


def test_product_bwd_refusals():
    L = lib()

    def bwd(name, d, dy=P[0], x=P[1], w=P[2], pre=P[3], dx=P[4], dw=P[5], db=P[6], flags=8, ws=P[7], n=1 << 33):
        return getattr(L, name)(d, dy, x, w, pre, dx, dw, db, flags, ws, n, None)
    for name in ("ssd_linear_bwd", "ssd_gated_bwd"):
        f = lambda d, **kw: bwd(name, d, **kw)
        assert f(None) == 1 and f(dims(dtype=7)) == 3 and f(dims(m=0)) == 2 and f(dims(m=1 << 31)) == 4
        assert f(dims(xs=-1)) == 2 and f(dims(gs=-1)) == 2 and f(dims(), flags=2) == 2
        for bad in (dict(dy=None), dict(x=None), dict(w=None), dict(pre=None), dict(dx=None, dw=None, db=None)):
            assert f(dims(), **bad) == 1, bad
        for bad in (dict(dy=P[0] + 2), dict(dx=P[4] + 1), dict(db=P[6] + 2), dict(ws=P[7] + 8)):
            assert f(dims(), **bad) == 5, bad
        for bad in (dict(dx=P[1]), dict(dw=P[2]), dict(db=P[0] + 4), dict(dx=P[5]), dict(ws=P[3])):
            assert f(dims(), **bad) == 8, bad
        assert f(dims(), n=16) == 6 and f(dims(), ws=None) == 6
    assert bwd("ssd_gated_bwd", dims(), flags=0) == 2
    need = L.ssd_linear_bwd_workspace_bytes(dims(), 0)
    assert 0 < need < L.ssd_linear_bwd_workspace_bytes(dims(), 8)   # without an activation dpre is dy
    assert bwd("ssd_linear_bwd", dims(), flags=0, pre=None, n=need - 1) == 6
    assert L.ssd_linear_bwd_workspace_bytes(dims(), 64) == 0 and L.ssd_linear_bwd_workspace_bytes(dims(k=0), 0) == 0
    assert L.ssd_gated_bwd_workspace_bytes(dims(k=0)) == 0


def rn_dims(rows=5, D=32, dtype=0, reserved=0, strides=None):
    return ssd.ResidualNormDims(rows, D, dtype, reserved, *(strides or [D] * 5))


def test_residual_norm_refusals():
    L = lib()

    def fwd(d, b=P[0], r=P[1], z=P[2], post=P[3], sc=P[4], pre=P[5], eps=1e-5, total=P[6], y=P[7], st=P[8]):
        return L.ssd_residual_norm_fwd(d, b, r, z, post, sc, pre, eps, total, y, st, None)
    assert fwd(None) == 1 and fwd(rn_dims(dtype=4)) == 3 and fwd(rn_dims(reserved=1)) == 2
    assert fwd(rn_dims(rows=0)) == 2 and fwd(rn_dims(D=0)) == 2 and fwd(rn_dims(D=1 << 30)) == 4 and fwd(rn_dims(rows=1 << 60)) == 2
    for bad in (dict(b=None), dict(total=None), dict(y=None), dict(pre=None)):
        assert fwd(rn_dims(), **bad) == 1, bad
    for eps in (-1.0, float("nan"), float("inf")):
        assert fwd(rn_dims(), eps=eps) == 2
    for k in range(3):
        s = [32] * 5
        s[k] = -1
        assert fwd(rn_dims(strides=s)) == 2
    assert fwd(rn_dims(strides=[32, -1, -1, -1, -1]), r=None, z=None, y=P[0]) == 8      # absent ones are not looked at
    assert fwd(rn_dims(), b=P[0] + 2) == 5 and fwd(rn_dims(), post=P[3] + 2) == 5
    for bad in (dict(total=P[0]), dict(y=P[1]), dict(y=P[6] + 4), dict(st=P[7]), dict(total=P[1] + 4), dict(total=P[3])):
        assert fwd(rn_dims(), **bad) == 8, bad
    assert fwd(rn_dims(strides=[32, 40, 32, 32, 32]), total=P[1]) == 8      # in place at a stride of its own
    assert fwd(rn_dims(), total=P[1], y=P[1]) == 8

    def bwd(d, dy=P[0], dt=P[1], b=P[2], r=P[3], z=P[4], post=P[5], sc=P[6], pre=P[7], st=P[8], db=P[9], dr=P[10], dz=P[11],
            dpost=P[12], dsc=P[13], dpre=P[14], ws=P[15], n=1 << 30):
        return L.ssd_residual_norm_bwd(d, dy, dt, b, r, z, post, sc, pre, st, db, dr, dz, dpost, dsc, dpre, ws, n, None)
    need = L.ssd_residual_norm_bwd_workspace_bytes(rn_dims())
    assert need > 0 and L.ssd_residual_norm_bwd_workspace_bytes(rn_dims(D=0)) == 0
    assert bwd(None) == 1 and bwd(rn_dims(), n=need - 1) == 6 and bwd(rn_dims(), ws=None) == 6
    for bad in (dict(b=None), dict(st=None), dict(db=None), dict(dy=None), dict(pre=None), dict(dz=None), dict(z=None),
                dict(dy=None, pre=None, dpre=None, dt=None), dict(r=None), dict(post=None), dict(sc=None)):
        assert bwd(rn_dims(), **bad) == 1, bad
    for bad in (dict(db=P[2]), dict(dr=P[1]), dict(dz=P[9]), dict(dpost=P[13] + 4), dict(ws=P[8])):
        assert bwd(rn_dims(), **bad) == 8, bad


def clip(n=2, ins=(P[0], P[1]), outs=(P[0], P[1]), sizes=(100, 7), codes=(0, 1), max_norm=1.0, norm=P[2], ws=P[3], b=1 << 20):
    L = lib()
    arr = lambda t, v: None if v is None else (t * max(len(v), 1))(*v)
    return L.ssd_clip(n, arr(ctypes.c_void_p, ins), arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, sizes),
                      arr(ctypes.c_int32, codes), max_norm, norm, ws, b, None)


def test_clip_refusals():
    L = lib()
    size = lambda *s: L.ssd_clip_workspace_bytes(len(s), (ctypes.c_int64 * len(s))(*s))
    assert size(100, 7) > 0 and size(0) > 0 and size(-1) == 0 and size(1 << 58, 1 << 58) == 0
    assert L.ssd_clip_workspace_bytes(0, None) == 0 and L.ssd_clip_workspace_bytes(1, None) == 0
    assert clip(n=0) == 2 and clip(sizes=(100, -7)) == 2 and clip(sizes=(1 << 58, 1 << 58)) == 2
    for bad in (dict(ins=None), dict(codes=None), dict(sizes=None), dict(norm=None), dict(ins=(P[0], None)),
                dict(outs=(None, P[1]))):
        assert clip(**bad) == 1, bad
    assert clip(codes=(0, 3)) == 3
    for m in (-1.0, float("nan")):
        assert clip(max_norm=m) == 2
    assert clip(b=8) == 6 and clip(ws=None) == 6
    for bad in (dict(ins=(P[0] + 2, P[1]), outs=(P[0] + 2, P[1])), dict(ins=(P[0], P[1] + 1), outs=(P[0], P[1] + 1)),
                dict(norm=P[2] + 2), dict(ws=P[3] + 8)):
        assert clip(**bad) == 5, bad
    for bad in (dict(ins=(P[0], P[0]), outs=(P[0], P[0])),                     # the same tensor twice, in place
                dict(ins=(P[0], P[0] + 396), outs=(P[0], P[0] + 396)),         # the last element of another
                dict(outs=(P[4], P[4] + 200)), dict(outs=(P[1], P[0])), dict(outs=(P[0] + 4, P[1])),
                dict(norm=P[0] + 8), dict(ws=P[1]), dict(norm=P[3])):
        assert clip(**bad) == 8, bad


# ------------------------------------------------------------------------------ binding
z = torch.zeros


@pytest.mark.parametrize("name,change,msg", [
    ("x", lambda t: t.half(), "x has dtype"), ("x", lambda t: t[0], "x has shape"), ("x", lambda t: None, "x must be"),
    ("x", lambda t: z(5, 16)[:, ::2], "x must have contiguous channels"),
    ("weight", lambda t: t.bfloat16(), "weight has dtype"), ("weight", lambda t: t[:, :7], "weight has shape"),
    ("weight", lambda t: z(8, 6).t(), "weight must be contiguous"), ("weight", lambda t: None, "weight must be"),
    ("bias", lambda t: t[:5], "bias has shape"), ("bias", lambda t: t.bfloat16(), "bias has dtype"),
    ("residual", lambda t: t[:4], "residual has shape"), ("residual", lambda t: t.bfloat16(), "residual has dtype"),
    ("act", lambda t: "relu", "act must be"), ("act", lambda t: [], "act must be"), ("x", lambda t: t, "CUDA device"),
])
def test_linear_binding(name, change, msg):
    lib()
    a = dict(x=z(5, 8), weight=z(6, 8), bias=z(6), residual=z(5, 6), act="silu")
    a[name] = change(a[name])
    with pytest.raises(ValueError, match=msg):
        ssd.linear_fwd(**a)
    if name != "residual":
        with pytest.raises(ValueError, match=msg):
            ssd.linear_bwd(z(5, 6), a["x"], a["weight"], a["bias"], z(5, 6), act=a["act"])
        if name != "act":
            with pytest.raises(ValueError, match=msg):
                ssd.gated_fwd(a["x"], a["weight"], a["bias"])


def test_product_binding_beside():
    lib()
    x, w = z(5, 8), z(6, 8)
    for call, msg in ((lambda: ssd.gated_fwd(x, z(7, 8)), "as many for g as for u"),
                      (lambda: ssd.linear_bwd(None, x, w), "dy must be"),
                      (lambda: ssd.linear_bwd(z(5, 5), x, w), "dy has shape"),
                      (lambda: ssd.linear_bwd(z(5, 6), x, w, act="gelu"), "pre"),
                      (lambda: ssd.linear_bwd(z(5, 6), x, w, None, z(5, 7), act="gelu"), "pre has shape"),
                      (lambda: ssd.gated_bwd(z(5, 6), x, w, None, z(5, 6)), "dh has shape"),
                      (lambda: ssd.gated_bwd(z(5, 3), x, w, None, None), "pre"),
                      (lambda: ssd.gated_bwd(z(5, 3), x, w, None, z(5, 3)), "pre has shape")):
        with pytest.raises(ValueError, match=msg):
            call()


@pytest.mark.parametrize("change,msg", [
    (dict(branch=z(3, 8, dtype=torch.float64)), "branch has dtype"), (dict(branch=z(8)), "branch has shape"),
    (dict(residual=z(3, 7)), "residual has shape"), (dict(gate=z(3, 8).bfloat16()), "gate has dtype"),
    (dict(gate=z(3, 16)[:, ::2]), "gate must have contiguous"), (dict(post_weight=z(7)), "post_weight has shape"),
    (dict(scale=z(8).bfloat16()), "scale has dtype"), (dict(pre_weight=z(16)[::2]), "pre_weight must be contiguous"),
    (dict(pre_weight=None, y=z(3, 8)), "y is given"), (dict(), "CUDA device"),
])
def test_residual_norm_binding(change, msg):
    lib()
    a = dict(branch=z(3, 8), residual=z(3, 8), gate=z(3, 8), post_weight=z(8), scale=z(8), pre_weight=z(8))
    a.update(change)
    with pytest.raises(ValueError, match=msg):
        ssd.residual_norm_fwd(**a)


def test_residual_norm_bwd_binding():
    lib()
    b, w, st = z(3, 8), z(8), z(2, 3)
    for call, msg in ((lambda: ssd.residual_norm_bwd(None, b, b, None, None, None, None, w, st), "dy has to be given"),
                      (lambda: ssd.residual_norm_bwd(b, b, b, None, None, None, None, None, st), "dy has to be given"),
                      (lambda: ssd.residual_norm_bwd(None, None, b, None, None, None, None, None, st), "both None"),
                      (lambda: ssd.residual_norm_bwd(b, None, b, None, None, None, None, w, z(3)), "stats has shape"),
                      (lambda: ssd.residual_norm_bwd(b, None, b, None, None, None, None, w, None), "stats")):
        with pytest.raises(ValueError, match=msg):
            call()


def test_clip_binding():
    lib()
    for call, msg in ((lambda: ssd.grad_norm([]), "no tensors"), (lambda: ssd.grad_norm([None]), "tensor 0 must be"),
                      (lambda: ssd.clip_grads([z(3), None], 1.0), "tensor 1 must be"),
                      (lambda: ssd.clip_grads([z(3), z(4).half()], 1.0), "tensor 1 has dtype"),
                      (lambda: ssd.clip_grads([z(3, 4).t()], 1.0), "tensor 0 must be contiguous"),
                      (lambda: ssd.clip_grads([z(3)], 1.0, out=[]), "out has 0"),
                      (lambda: ssd.clip_grads([z(3)], 1.0, out=[z(4)]), "out 0 must be"),
                      (lambda: ssd.clip_grads([z(3)], 1.0, out=[z(3).bfloat16()]), "out 0 must be"),
                      (lambda: ssd.clip_grads([z(3)], 1.0, out=[None]), "out 0 must be"),
                      (lambda: ssd.clip_grads([z(3)], 1.0), "CUDA device")):
        with pytest.raises(ValueError, match=msg):
            call()


# ------------------------------------------------------- versions of written tensors, no library
class _Library:
    """Every entry point succeeds; sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_bytes") else 0


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(ssd, "lib", lambda: _Library())
    monkeypatch.setattr(ssd, "_elsewhere", lambda t, stream: None)
    monkeypatch.setattr(ssd, "_current", lambda t: 0)


def test_written_tensors_have_a_new_version(no_library):
    y, h, total, n = z(5, 6), z(5, 3), z(5, 8), z(5, 8)
    ssd.linear_fwd(z(5, 8), z(6, 8), y=y)
    ssd.gated_fwd(z(5, 8), z(6, 8), h=h)
    ssd.residual_norm_fwd(z(5, 8), pre_weight=z(8), y=n, total=total)
    g, out = [z(3), z(4)], [z(3), z(4)]
    ssd.clip_grads(g, 1.0, out=out)
    assert all(t._version == 1 for t in (y, h, total, n, *out)) and all(t._version == 0 for t in g)
    ssd.clip_grads(g, 1.0)
    ssd.grad_norm(out)
    assert all(t._version == 1 for t in g + out)


def test_backward_after_its_residual_was_written_raises(no_library):
    from chunked_linear_recurrence_amd import block
    b, r = z(5, 8).requires_grad_(True), z(5, 8)
    y, total = block.residual_norm(b, r, pre_weight=z(8))
    ssd.residual_norm_fwd(z(5, 8), r, total=r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
