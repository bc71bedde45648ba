"""Plain float64 references of a layer's feed-forward half, from their definitions, and bounds of
what a kernel may be off by, value by value.

Roundings counted: h = half a step of the activations' type, relative (0 where it is float32),
for each value that is stored in it; 2^-23 for each of K + 4 additions of a float32 sum, relative
to the sum of the terms' sizes (twice half a step, as the matrix units' own order and rounding
are not ours); 2^-20 for the float32 activations, of their value or of 1 for a derivative."""
import torch

F64 = torch.float64
U = 2.0 ** -23
ACT = 2.0 ** -20


def half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def up(t):
    return None if t is None else t.detach().cpu().to(F64)


def ndtr(v):
    """Phi(v) with its tail's relative accuracy (1 + erf keeps steps of 2^-54)."""
    return 0.5 * torch.special.erfc(-v * 2.0 ** -0.5)


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * ndtr(v)
    return v


def dact(v, name):
    if name == "silu":
        s = torch.sigmoid(v)
        return s + v * s * (1 - s)
    if name == "gelu":
        return ndtr(v) + v * torch.exp(-v * v / 2) * (2 * torch.pi) ** -0.5
    return torch.ones_like(v)


CURVE = {None: 0.0, "silu": 0.5, "gelu": 0.8}      # the largest |act''|
SLOPE = {None: 1.0, "silu": 1.1, "gelu": 1.13}     # the largest |act'|


def inside(got, ref, bound, what):
    g = up(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), what + " has values that are not finite"
    over = (g - ref).abs() - bound
    assert (over <= 0).all(), "%s: off by %.3g where %.3g is allowed (value %.3g)" % (
        what, (g - ref).abs().flatten()[over.argmax()], bound.flatten()[over.argmax()], ref.flatten()[over.argmax()])


def check_linear(dtype, got, x, w, bias, residual, name, dy=None):
    """got: (y, pre or None) or with dy (y, pre, dx, dweight, dbias)."""
    h, k = half(dtype), x.shape[1]
    X, W = up(x), up(w)
    B = torch.zeros(W.shape[0], dtype=F64) if bias is None else up(bias)
    R = torch.zeros(1, 1, dtype=F64) if residual is None else up(residual)
    pre = X @ W.t() + B
    size = X.abs() @ W.abs().t() + B.abs()
    e_pre = (k + 4) * U * size
    y = act(pre, name) + R
    e = SLOPE[name] * e_pre + ACT * act(pre, name).abs() + U * y.abs() + 1e-30
    inside(got[0], y, e * (1 + h) + h * y.abs(), "y")
    if got[1] is not None:
        inside(got[1], pre, e_pre * (1 + h) + h * pre.abs(), "pre")
    if dy is None:
        return
    G = up(dy)
    d = G * dact(pre, name)
    e_d = torch.zeros_like(d)
    if name is not None:
        e_d = G.abs() * (CURVE[name] * (e_pre * (1 + h) + h * pre.abs()) + ACT)
    check_grads(dtype, got[2:], X, W, d, e_d, e_d + (h * (d.abs() + e_d) if name is not None else 0.0), bias is not None)


def check_gated(dtype, got, x, w, bias, name, dh=None):
    """got: (h, pre or None) or with dh (h, pre, dx, dweight, dbias)."""
    r, k, f = half(dtype), x.shape[1], w.shape[0] // 2
    X, W = up(x), up(w)
    B = torch.zeros(2 * f, dtype=F64) if bias is None else up(bias)
    pre = X @ W.t() + B
    e_pre = (k + 4) * U * (X.abs() @ W.abs().t() + B.abs())
    g, u, eg, eu = pre[:, :f], pre[:, f:], e_pre[:, :f], e_pre[:, f:]
    a = act(g, name)
    ea = SLOPE[name] * eg + ACT * a.abs()
    y = a * u
    e = ea * u.abs() + a.abs() * eu + ea * eu + U * y.abs() + 1e-30
    inside(got[0], y, e * (1 + r) + r * y.abs(), "h")
    if got[1] is not None:
        inside(got[1], pre, e_pre * (1 + r) + r * pre.abs(), "pre")
    if dh is None:
        return
    G = up(dh)
    kept = e_pre * (1 + r) + r * pre.abs()                 # what the kept values are off by
    kg, ku = kept[:, :f], kept[:, f:]
    s = dact(g, name)
    es = CURVE[name] * kg + ACT
    dg, du = G * u * s, G * a
    e_g = G.abs() * (u.abs() * es + ku * s.abs() + ku * es) + 2 * U * dg.abs()
    e_u = G.abs() * (SLOPE[name] * kg + ACT * a.abs()) + 2 * U * du.abs()
    d, e_d = torch.cat([dg, du], 1), torch.cat([e_g, e_u], 1)
    check_grads(dtype, got[2:], X, W, d, e_d, e_d + r * (d.abs() + e_d), bias is not None)


def check_grads(dtype, got, X, W, d, e_sum, e_d, has_bias):
    """dx, dweight and dbias from dpre = d, known to e_sum before and e_d after it is rounded."""
    h = half(dtype)
    m, n = d.shape

    def bound(ref, e):
        return e * (1 + h) + h * ref.abs() + 1e-30
    if got[0] is not None:
        dx = d @ W
        inside(got[0], dx, bound(dx, e_d @ W.abs() + (n + 4) * U * ((d.abs() + e_d) @ W.abs())), "dx")
    if got[1] is not None:
        dw = d.t() @ X
        inside(got[1], dw, bound(dw, e_d.t() @ X.abs() + (m + 4) * U * ((d.abs() + e_d).t() @ X.abs())), "dweight")
    assert (got[2] is not None) == has_bias
    if has_bias:
        db = d.sum(0)
        inside(got[2], db, bound(db, e_sum.sum(0) + (m + 4) * U * (d.abs() + e_sum).sum(0)), "dbias")
