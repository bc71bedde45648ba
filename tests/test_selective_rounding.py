"""The selective scan within bounds that follow its roundings, value by value, against float64.

With e = 2^-24 (one float32 rounding) and 2^-22 for a hardware 2^x (twice its 1 ulp):

  step size   the argument delta + bias is rounded, scaled and summed: 4 e (|delta| + |bias|); the
              softplus itself (2^x, log2, a correction) 2^-20 of its value, several times its parts
  decay       relative: |A| times the step size's error, 64 e |dt A| for its product and the sum of
              a chunk's step sizes (chunks of at most 64 tokens here), 2^-22
  gate        relative: 2^-20 + 4 e |z|
  state       E_t = a E_{t-1} + |a h_{t-1}| (decay's) + |dt u B| (step size's, 6 e) + 2 e |h|

and so on through the formulas: a product adds its factors' relative errors and a few e, a sum its
terms' errors and e for each term's addition.  Second-order terms are covered by a factor of 1.05.
Results stored in bfloat16 are rounded once more (2^-8)."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd
from test_selective import make, on_gpu, reference, views

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
KEYS = ("u", "delta", "A", "B", "C", "D", "z", "bias")


def within(got, ref, bound, dtype, what):
    g, r = R.up(got), ref.detach()
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (r.abs() + bound)
    else:
        bound = bound + 2 * E * r.abs()
    over = ((g - r).abs() / bound.clamp(min=1e-30)).max()
    assert torch.isfinite(g).all() and over <= 1, "%s: %.3g times its bound" % (what, over)


def bounds(t, softplus):
    """Bounds of the errors of y, final_state and every gradient (by the input's name)."""
    u, delta, A, B, C, D, z, bias, st, dy, df = (R.up(t[k]) for k in KEYS + ("st", "dy", "df"))
    b, L, d = u.shape
    G, N = B.shape[2:]
    grp = torch.arange(d) // (d // G)
    raw = delta + bias
    size = 4 * E * (delta.abs() + bias.abs())                     # the argument's error
    dt = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    sig = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    dt_err = sig * size + (2.0 ** -20 * dt if softplus else 0)
    sig_err = sig * (2.0 ** -20 + size) if softplus else torch.zeros_like(sig)
    s = torch.sigmoid(z)
    gate, gate_rel = z * s, 2.0 ** -20 + 4 * E * z.abs()
    dgate = s * (1 + z * (1 - s))
    dgate_err = s * (1 + z.abs() * (1 - s)) * 2 * gate_rel
    over_d = lambda v: v.unflatten(1, (G, -1)).sum(2)             # channels of a group

    h, Eh = st, torch.zeros_like(st)
    hs, Ehs, decays, rels, y0, Ey0 = [h], [Eh], [], [], [], []
    for k in range(L):
        Bk, Ck = B[:, k][:, grp], C[:, k][:, grp]
        a = torch.exp(dt[:, k, :, None] * A)
        rel = A.abs() * dt_err[:, k, :, None] + 64 * E * (dt[:, k, :, None] * A).abs() + 2.0 ** -22
        x = (dt[:, k] * u[:, k])[..., None] * Bk
        x_err = (dt_err[:, k] * u[:, k].abs())[..., None] * Bk.abs() + 6 * E * x.abs()
        Eh = a * Eh + (a * h).abs() * rel + x_err
        h = a * h + x
        Eh = Eh + 2 * E * h.abs()
        y0.append((Ck * h).sum(-1) + D * u[:, k])
        Ey0.append((Ck.abs() * Eh).sum(-1) + (N + 6) * E * (Ck * h).abs().sum(-1) + 4 * E * (D * u[:, k]).abs())
        for seq, v in ((hs, h), (Ehs, Eh), (decays, a), (rels, rel)):
            seq.append(v)
    y0, Ey0 = torch.stack(y0, 1), torch.stack(Ey0, 1)
    out = {"y": Ey0 * gate.abs() + (y0 * gate).abs() * (gate_rel + 4 * E), "final_state": Eh}

    r = dy * gate
    r_err = r.abs() * (gate_rel + 2 * E)
    out["z"] = (dy * dgate).abs() * Ey0 + (dy * y0).abs() * (dgate_err + 4 * E * dgate.abs())
    out["D"] = (r_err * u.abs() + (b * L + 4) * E * (r * u).abs()).sum((0, 1))
    for key, like in (("u", u), ("delta", u), ("B", B), ("C", C), ("A", A)):
        out[key] = torch.zeros_like(like)
    carry, Ec = df, torch.zeros_like(df)
    terms, ddelta = torch.zeros_like(A), torch.zeros_like(u)
    for k in reversed(range(L)):
        Bk, Ck, a, rel = B[:, k][:, grp], C[:, k][:, grp], decays[k], rels[k]
        rk, dtk, uk = r[:, k, :, None], dt[:, k], u[:, k]
        g = Ck * rk + carry
        Eg = Ck.abs() * r_err[:, k, :, None] + Ec + E * ((Ck * rk).abs() + g.abs())
        q, Eq = (g * Bk).sum(-1), (Bk.abs() * Eg).sum(-1) + (N + 2) * E * (g * Bk).abs().sum(-1)
        w = a * g * hs[k]
        Ew = w.abs() * (rel + 4 * E) + (a * hs[k]).abs() * Eg + (a * g).abs() * Ehs[k]
        Dr = D * r[:, k]
        out["u"][:, k] = dtk * Eq + dt_err[:, k] * q.abs() + D.abs() * r_err[:, k] + 4 * E * ((dtk * q).abs() + Dr.abs())
        dd = uk * q + (A * w).sum(-1)
        Ed = uk.abs() * Eq + (A.abs() * Ew).sum(-1) + (N + 4) * E * ((uk * q).abs() + (A * w).abs().sum(-1))
        ddelta[:, k] = dd * sig[:, k]
        out["delta"][:, k] = sig[:, k] * Ed + dd.abs() * (sig_err[:, k] + 2 * E)
        out["A"] += (dtk[..., None] * Ew + dt_err[:, k, :, None] * w.abs()).sum(0)
        terms += (dtk[..., None] * w).abs().sum(0)
        x = (dtk * uk)[..., None]
        x_err = (dt_err[:, k] * uk.abs())[..., None] + 4 * E * x.abs()
        out["B"][:, k] = over_d(Eg * x.abs() + g.abs() * x_err + (d + 6) * E * (g * x).abs())
        here, Ehere = hs[k + 1], Ehs[k + 1]
        out["C"][:, k] = over_d(rk.abs() * Ehere + here.abs() * r_err[:, k, :, None] + (d + 6) * E * (rk * here).abs())
        carry, Ec = a * g, a * Eg + (a * g).abs() * (rel + 2 * E)
    out["A"] += (b * L + 4) * E * terms
    out["st"] = Ec
    out["bias"] = (out["delta"] + (b * L + 4) * E * ddelta.abs()).sum((0, 1))
    return {k: 1.05 * v for k, v in out.items()}


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 48, 70, 16, 1), (1, 61, 130, 32, 2), (2, 40, 64, 64, 1), (1, 20, 200, 16, 2)], ids=str)
def test_errors_follow_the_roundings(shape, dtype, softplus):
    b, L, d, N, G = shape
    t = make(b, L, d, N, G, dtype, seed=41 + L)
    if not softplus:
        t["delta"] = (t["delta"].abs() * 0.1).to(dtype)
        t["bias"] = t["bias"].exp()
    g, t = on_gpu(t), views(t)
    y, f, kept = ssd.selective_fwd(*(g[k] for k in KEYS), g["st"], softplus=softplus, keep=True)
    r = ssd.selective_bwd(g["dy"], *(g[k] for k in KEYS), kept, dfinal=g["df"], softplus=softplus)
    torch.cuda.synchronize()
    yr, fr, gr = reference(t, ("D", "z", "bias", "st"), softplus)
    err = bounds(t, softplus)
    within(y, yr, err["y"], dtype, "y")
    within(f, fr, err["final_state"], torch.float32, "final_state")
    f32 = torch.float32
    for got, key, ty in ((r.du, "u", dtype), (r.ddelta, "delta", dtype), (r.dz, "z", dtype), (r.dB, "B", dtype),
                         (r.dC, "C", dtype), (r.dA, "A", f32), (r.dD, "D", f32), (r.ddelta_bias, "bias", f32),
                         (r.dinit, "st", f32)):
        within(got, gr[key], err[key], ty, "gradient of " + key)
