"""What the operators around a scan refuse (no GPU: every call fails before anything is
enqueued): the C ABI's status codes, and the binding's tensor checks."""
import ctypes

import pytest
import torch

from chunked_linear_recurrence_amd import ssd

F = 1 << 40                        # an aligned address that is never dereferenced
P = [F + (k << 34) for k in range(32)]


def lib():
    try:
        return ssd.lib()
    except RuntimeError:
        pytest.skip("libssdscan.so not built")


# ------------------------------------------------------------------------------- C ABI
def conv_dims(b=2, L=40, C=16, W=4, dtype=0, xs=None):
    xs = xs or (L * C, C)
    return ssd.ConvDims(b, L, C, W, dtype, xs[0], xs[1], L * C, C)


def conv_fwd(d, x=P[0], w=P[1], bias=P[2], init=P[3], lengths=P[4], y=P[5], fin=P[6], flags=8):
    return lib().ssd_conv_fwd(d, x, w, bias, init, lengths, y, fin, flags, None)


def test_conv_fwd_refusals():
    assert conv_fwd(None) == 1
    assert conv_fwd(conv_dims(dtype=2)) == 3
    for bad in (dict(b=0), dict(L=0), dict(C=0), dict(W=0), dict(xs=(-1, 16)), dict(xs=(640, -16)),
                dict(b=1 << 40, L=1 << 29, C=1 << 20)):
        assert conv_fwd(conv_dims(**bad)) == 2, bad
    for bad in (dict(W=1), dict(W=5), dict(L=1 << 31), dict(C=1 << 30)):
        assert conv_fwd(conv_dims(**bad)) == 4, bad
    for bad in (dict(x=None), dict(w=None), dict(y=None)):
        assert conv_fwd(conv_dims(), **bad) == 1, bad
    assert conv_fwd(conv_dims(), flags=1) == 2
    for bad in (dict(x=P[0] + 2), dict(w=P[1] + 1), dict(lengths=P[4] + 2), dict(y=P[5] + 2)):
        assert conv_fwd(conv_dims(), **bad) == 5, bad
    assert conv_fwd(conv_dims(dtype=1), x=P[0] + 1) == 5
    for bad in (dict(y=P[0] + 64), dict(fin=P[3] + 4), dict(fin=P[5] + 4), dict(y=P[1])):
        assert conv_fwd(conv_dims(), **bad) == 8, bad
    assert lib().ssd_last_error_message().decode() != ""
    # more workgroups than a grid holds
    assert conv_fwd(conv_dims(b=1 << 30, L=1, C=1 << 20, xs=(0, 0)), init=None, fin=None, y=1 << 6, x=1 << 62, w=1 << 61,
                    bias=None, lengths=None) == 4


def test_conv_step_refusals():
    step = lambda d, x=P[0], si=P[1], so=P[1], y=P[2], flags=0: lib().ssd_conv_step(d, x, P[3], None, si, so, y, flags, None)
    assert step(conv_dims()) == 2                       # not one token
    d = conv_dims(L=1)
    assert step(d, si=None) == 1 and step(d, so=None) == 1 and step(d, y=None) == 1
    assert step(d, so=P[1] + 8) == 8 and step(d, y=P[1]) == 8
    assert step(d, flags=16) == 2


def test_conv_bwd_refusals():
    L = lib()

    def bwd(d, dy=P[0], x=P[1], dx=P[2], dw=P[3], db=P[4], di=P[5], ws=P[6], n=1 << 20, flags=0):
        return L.ssd_conv_bwd(d, dy, x, P[7], P[8], P[9], P[10], P[11], dx, dw, db, di, flags, ws, n, None)
    d = conv_dims()
    need = L.ssd_conv_bwd_workspace_bytes(d)
    assert need > 0 and L.ssd_conv_bwd_workspace_bytes(conv_dims(W=7)) == 0
    assert bwd(d, n=need - 1) == 6 and bwd(d, ws=None) == 6
    assert bwd(d, dx=None) == 1 and bwd(d, dw=None) == 1
    assert bwd(d, dx=P[1]) == 8 and bwd(d, ws=P[2]) == 8 and bwd(d, di=P[9]) == 8
    assert bwd(d, flags=2) == 2


def sel_dims(b=2, L=40, D=64, N=16, G=1, dtype=0, reserved=0, over=None):
    s = [L * D, D] * 3 + [L * G * N, G * N] * 2 + [L * D, D]
    for k, v in (over or {}).items():
        s[k] = v
    return ssd.SelectiveDims(b, L, D, N, G, dtype, reserved, *s)


def sel_fwd(d, u=P[0], delta=P[1], A=P[2], B=P[3], C=P[4], D=P[5], z=P[6], bias=P[7], init=P[8], lengths=P[9], y=P[10],
            fin=P[11], kept=P[12], flags=16, ws=P[13], n=1 << 33):
    return lib().ssd_selective_fwd(d, u, delta, A, B, C, D, z, bias, init, lengths, y, fin, kept, flags, ws, n, None)


def test_selective_fwd_refusals():
    assert sel_fwd(None) == 1
    assert sel_fwd(sel_dims(dtype=-1)) == 3
    for bad in (dict(b=0), dict(L=0), dict(D=0), dict(N=0), dict(G=0), dict(D=66, G=4), dict(reserved=1),
                dict(over={0: -1}), dict(over={7: -2}), dict(b=1 << 40, L=1 << 29, D=1 << 20)):
        assert sel_fwd(sel_dims(**bad)) == 2, bad
    for bad in (dict(N=8), dict(N=24), dict(N=128), dict(L=1 << 31), dict(D=1 << 24)):
        assert sel_fwd(sel_dims(**bad)) == 4, bad
    for name in ("u", "delta", "A", "B", "C", "y"):
        assert sel_fwd(sel_dims(), **{name: None}) == 1, name
    assert sel_fwd(sel_dims(), flags=8) == 2
    for bad in (dict(u=P[0] + 2), dict(B=P[3] + 2), dict(kept=P[12] + 8), dict(ws=P[13] + 8)):
        assert sel_fwd(sel_dims(), **bad) == 5, bad
    assert sel_fwd(sel_dims(dtype=1), B=P[3] + 2) == 5           # bfloat16 rows of B and C on 4 bytes
    assert sel_fwd(sel_dims(dtype=1, over={7: 17})) == 5
    assert sel_fwd(sel_dims(dtype=1, over={8: 641})) == 5
    d = sel_dims()
    need = lib().ssd_selective_fwd_workspace_bytes(d)
    assert sel_fwd(d, n=need - 1) == 6 and sel_fwd(d, ws=None) == 6
    for bad in (dict(y=P[0]), dict(y=P[6] + 4), dict(fin=P[8] + 64), dict(kept=P[10]), dict(ws=P[1]), dict(ws=P[12])):
        assert sel_fwd(d, **bad) == 8, bad


def test_selective_step_refusals():
    L = lib()

    def step(d, si=P[8], so=P[8], y=P[9], u=P[0]):
        return L.ssd_selective_step(d, u, P[1], P[2], P[3], P[4], P[5], P[6], P[7], si, so, y, 16, None)
    assert step(sel_dims()) == 2
    d = sel_dims(L=1)
    assert step(d, si=None) == 1 and step(d, so=None) == 1 and step(d, u=None) == 1
    assert step(d, si=P[8] + 4) == 5 and step(d, so=P[10] + 4) == 5
    assert step(d, so=P[8] + 16) == 8 and step(d, y=P[8]) == 8 and step(d, y=P[6]) == 8


def test_selective_bwd_refusals():
    L = lib()

    def bwd(d, z=P[6], kept=P[8], du=P[11], dz=P[17], dA=P[13], ws=P[20], n=1 << 33, flags=16):
        return L.ssd_selective_bwd(d, P[0], P[1], P[2], P[3], P[4], P[5], P[7], z, P[21], kept, P[9], P[10], du, P[12], dA,
                                   P[14], P[15], P[16], dz, P[18], P[19], flags, ws, n, None)
    d = sel_dims()
    need = L.ssd_selective_bwd_workspace_bytes(d)
    assert need > 0 and L.ssd_selective_kept_bytes(d) == 2 * 5 * 1 * 16 * 64 * 4
    assert L.ssd_selective_bwd_workspace_bytes(sel_dims(N=5)) == 0 and L.ssd_selective_kept_bytes(sel_dims(N=5)) == 0
    assert bwd(d, n=need - 1) == 6 and bwd(d, ws=None) == 6
    assert bwd(d, kept=None) == 1 and bwd(d, du=None) == 1 and bwd(d, dA=None) == 1
    assert bwd(d, dz=None) == 1 and bwd(d, z=None) == 1          # dz exactly if z
    assert bwd(d, du=P[0]) == 8 and bwd(d, ws=P[8]) == 8 and bwd(d, dA=P[3]) == 8
    assert bwd(d, flags=1) == 2


def test_norm_refusals():
    L = lib()
    dims = lambda rows=4, D=32, dtype=0, reserved=0, xs=32: ssd.NormDims(rows, D, dtype, reserved, xs, 32)
    fwd = lambda d, x=P[0], y=P[1], eps=1e-5, m=P[2]: L.ssd_norm_fwd(d, x, P[3], P[4], eps, y, m, P[5], None)
    assert fwd(None) == 1 and fwd(dims(dtype=9)) == 3 and fwd(dims(reserved=2)) == 2
    assert fwd(dims(rows=0)) == 2 and fwd(dims(D=0)) == 2 and fwd(dims(xs=-1)) == 2 and fwd(dims(rows=1 << 60)) == 2
    assert fwd(dims(D=1 << 31)) == 4
    assert fwd(dims(), x=None) == 1 and fwd(dims(), y=None) == 1
    assert fwd(dims(), eps=-1.0) == 2 and fwd(dims(), eps=float("nan")) == 2 and fwd(dims(), eps=float("inf")) == 2
    assert fwd(dims(), x=P[0] + 2) == 5 and fwd(dims(), y=P[0] + 4) == 8 and fwd(dims(), m=P[1]) == 8
    bwd = lambda d, dx=P[3], ws=P[6], n=1 << 20, mean=P[4]: L.ssd_norm_bwd(d, P[0], P[1], P[2], mean, P[5], dx, P[7], P[8],
                                                                         ws, n, None)
    need = L.ssd_norm_bwd_workspace_bytes(dims())
    assert need > 0 and L.ssd_norm_bwd_workspace_bytes(dims(D=0)) == 0
    assert bwd(dims(), n=need - 1) == 6 and bwd(dims(), mean=None) == 1 and bwd(dims(), dx=P[0]) == 8
    assert bwd(dims(), ws=P[1]) == 8


# ------------------------------------------------------------------------------ binding
def _conv():
    return dict(x=torch.zeros(2, 9, 8), weight=torch.zeros(8, 4), bias=torch.zeros(8), init_state=torch.zeros(2, 3, 8),
                lengths=torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("name,change,msg", [
    ("x", lambda t: t.half(), "x has dtype"),
    ("x", lambda t: t[0], "x has shape"),
    ("x", lambda t: torch.zeros(2, 9, 16)[..., ::2], "x must have contiguous channels"),
    ("weight", lambda t: t.bfloat16(), "weight has dtype"),
    ("weight", lambda t: t[:7], "weight has shape"),
    ("weight", lambda t: torch.zeros(4, 8).t(), "weight must be contiguous"),
    ("bias", lambda t: t[:5], "bias has shape"),
    ("init_state", lambda t: t[:, :2], "init_state has shape"),
    ("init_state", lambda t: t.bfloat16(), "init_state has dtype"),
    ("lengths", lambda t: t.long(), "lengths has dtype"),
    ("x", lambda t: t, "CUDA device"),
])
def test_conv_binding(name, change, msg):
    lib()
    a = _conv()
    a[name] = change(a[name])
    with pytest.raises(ValueError, match=msg):
        ssd.conv_fwd(a["x"], a["weight"], a["bias"], a["init_state"], lengths=a["lengths"])
    if name != "lengths":
        with pytest.raises(ValueError, match=msg):
            ssd.conv_bwd(torch.zeros_like(a["x"]), a["x"], a["weight"], a["bias"], a["init_state"])


def _sel():
    b, L, d, N, G = 2, 9, 8, 16, 2
    z = lambda *s: torch.zeros(*s)
    return dict(u=z(b, L, d), delta=z(b, L, d), A=z(d, N), B=z(b, L, G, N), C=z(b, L, G, N), D=z(d), z=z(b, L, d),
                delta_bias=z(d), init_state=z(b, d, N))


@pytest.mark.parametrize("name,change,msg", [
    ("u", lambda t: t.double(), "u has dtype"),
    ("delta", lambda t: t.bfloat16(), "delta has dtype"),
    ("delta", lambda t: t[:, :8], "delta has shape"),
    ("A", lambda t: t[:, :8], "A has shape"),
    ("A", lambda t: t.bfloat16(), "A has dtype"),
    ("B", lambda t: t[:, :, 0], "B has shape"),
    ("B", lambda t: torch.zeros(2, 9, 2, 32)[..., :16], "B must have contiguous groups"),
    ("C", lambda t: t[:, :, :1], "C has shape"),
    ("C", lambda t: t.bfloat16(), "C has dtype"),
    ("z", lambda t: torch.zeros(2, 9, 16)[..., ::2], "z must have contiguous channels"),
    ("D", lambda t: t[:3], "D has shape"),
    ("delta_bias", lambda t: t.double(), "delta_bias has dtype"),
    ("init_state", lambda t: t[:, :, :8], "init_state has shape"),
    ("u", lambda t: t, "CUDA device"),
])
def test_selective_binding(name, change, msg):
    lib()
    a = _sel()
    a[name] = change(a[name])
    with pytest.raises(ValueError, match=msg):
        ssd.selective_fwd(**a)


def test_step_and_norm_binding():
    lib()
    with pytest.raises(ValueError, match="state has shape"):
        ssd.conv_step(torch.zeros(2, 8), torch.zeros(8, 4), None, torch.zeros(2, 4, 8))
    s = _sel()
    step = [s[k][:, 0] for k in ("u", "delta")] + [s["A"], s["B"][:, 0], s["C"][:, 0], s["D"], s["z"][:, 0], s["delta_bias"]]
    with pytest.raises(ValueError, match="state has dtype"):
        ssd.selective_step(*step, s["init_state"].bfloat16())
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.selective_step(*step, s["init_state"])
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="weight has shape"):
        ssd.norm_fwd(x, torch.zeros(7))
    with pytest.raises(ValueError, match="x has shape"):
        ssd.norm_fwd(torch.zeros(1, 3, 8))
    with pytest.raises(ValueError, match="mean has shape"):
        ssd.norm_bwd(x, x, None, torch.zeros(2), torch.zeros(3))
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.norm_fwd(x)


def test_selective_bwd_needs_the_forward_s_kept_states():
    lib()
    s = _sel()
    with pytest.raises(ValueError, match="kept has shape"):
        ssd.selective_bwd(torch.zeros(2, 9, 8), s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                          torch.zeros(16, dtype=torch.uint8))


def test_missing_tensors_are_named():
    lib()
    a, s = _conv(), _sel()
    for call, msg in ((lambda: ssd.conv_fwd(None, a["weight"]), "x must be"),
                      (lambda: ssd.conv_fwd(a["x"], None), "weight must be"),
                      (lambda: ssd.conv_bwd(None, a["x"], a["weight"]), "dy must be"),
                      (lambda: ssd.selective_fwd(s["u"], None, s["A"], s["B"], s["C"]), "delta must be"),
                      (lambda: ssd.selective_fwd(s["u"], s["delta"], s["A"], None, s["C"]), "B must be"),
                      (lambda: ssd.norm_bwd(None, a["x"][0], None, None, None), "dy must be")):
        with pytest.raises(ValueError, match=msg):
            call()


def test_strides_of_absent_tensors_are_not_looked_at():
    """z's and dy's strides mean nothing without them, and a step has no token strides."""
    d = sel_dims(over={4: -1, 5: -1, 10: -1, 11: -1})
    assert sel_fwd(d, z=None, n=0) == 6                       # past the strides: the workspace
    assert sel_fwd(d, n=0) == 2
    one = sel_dims(L=1, dtype=1, over={1: -1, 7: 3})
    assert lib().ssd_selective_step(one, P[0], P[1], P[2], P[3] + 2, P[4], P[5], P[6], P[7], P[8] + 4, P[8], P[9], 16, None) == 5
