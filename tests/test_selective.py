"""The selective scan (selective_fwd, selective_step, selective_bwd) against float64.

Tolerance: one step rounds a state about 4 times (decay, its exponent, product, sum; 2^-24
each) and an error lives as long as the state's memory, at most the tokens of a test (600):
600 * 4 * 2^-24 = 1.4e-4 of the largest value, if every rounding went the same way.  The
sums over states, channels and tokens add far less.  2e-4 of the largest value."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 2e-4
ACT = ("u", "delta", "B", "C", "z")


def make(b, L, d, N, G, dtype, seed, init=True, ragged=False, pad=None, extra=0):
    """Inputs on the CPU.  extra > 0: u, z, B and C are views into wider rows."""
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)
    t = dict(uz=randn(b, L, 2 * d + extra).to(dtype), delta=(randn(b, L, d) * 0.5).to(dtype),
             bc=randn(b, L, extra + 2 * G * N).to(dtype), D=torch.rand(d, generator=g),
             A=-(torch.arange(1, N + 1).float() * torch.exp(0.1 * randn(d, N))),
             st=randn(b, d, N) * 0.3 if init else None, dy=randn(b, L, d).to(dtype), df=randn(b, d, N))
    dt0 = torch.exp(torch.rand(d, generator=g) * 4.6 - 6.9)
    t["bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    t["lengths"] = None
    if ragged:
        t["lengths"] = torch.randint(0, L + 1, (b,), generator=g, dtype=torch.int32)
        t["lengths"][0], t["lengths"][-1] = L, 0
        for i in range(b):
            if pad is not None:
                for k in ("uz", "delta", "bc", "dy"):
                    t[k][i, int(t["lengths"][i]):] = pad
    t["d"], t["N"], t["G"], t["extra"] = d, N, G, extra
    return t


def views(t):
    d, N, G, e = t["d"], t["N"], t["G"], t["extra"]
    t["u"], t["z"] = t["uz"][..., :d], t["uz"][..., d + e:]
    t["B"] = t["bc"][..., e:e + G * N].unflatten(-1, (G, N))
    t["C"] = t["bc"][..., e + G * N:].unflatten(-1, (G, N))
    return t


def on_gpu(t):
    return views({k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in t.items()})


def reference(t, use, softplus, want=True):
    """Outputs and gradients in float64; `use` names the optional inputs in the call."""
    v = {k: R.up(t[k]) for k in ("u", "delta", "A", "B", "C")}
    for k in ("D", "z", "bias", "st"):
        v[k] = R.up(t[k]) if k in use and t[k] is not None else None
    leaves = {k: x.requires_grad_(want) for k, x in v.items() if x is not None}
    y, f = R.scan(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], v["bias"], v["st"], t["lengths"], softplus)
    if not want:
        return y, f, {}
    g = R.grads((y, f), (torch.nan_to_num(R.up(t["dy"])), R.up(t["df"])), list(leaves.values()))
    return y.detach(), f.detach(), dict(zip(leaves, g))


SHAPES = [  # b, L, D, N, G, init, ragged, extra
    (1, 1, 1, 16, 1, False, False, 0), (1, 1, 64, 16, 1, True, False, 0), (2, 7, 65, 16, 1, True, True, 2),
    (1, 8, 64, 32, 1, True, False, 0), (2, 9, 130, 16, 2, True, True, 6), (1, 16, 256, 16, 1, False, False, 0),
    (2, 17, 63, 64, 1, True, True, 0), (1, 31, 300, 16, 1, True, False, 8), (3, 64, 128, 32, 2, False, True, 4),
    (2, 100, 321, 16, 1, True, True, 0), (1, 257, 70, 64, 2, True, False, 2), (2, 600, 40, 16, 1, True, True, 10),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, dtype):
    b, L, d, N, G, init, ragged, extra = shape
    t = make(b, L, d, N, G, dtype, seed=L + d, init=init, ragged=ragged, extra=extra,
             pad=float("nan") if L % 2 else float("inf"))
    g = on_gpu(t)
    t = views(t)
    y, f, kept = ssd.selective_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], g["st"],
                                   lengths=g["lengths"], keep=True)
    y2, f2 = ssd.selective_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], g["st"],
                               lengths=g["lengths"])
    r = ssd.selective_bwd(g["dy"], g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], kept,
                          dfinal=g["df"], lengths=g["lengths"])
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(f, f2)
    yr, fr, gr = reference(t, ("D", "z", "bias", "st"), True)
    R.check(y, yr, dtype, TOL, "y")
    R.check(f, fr, torch.float32, TOL, "final_state")
    for name, got, key, ty in (("du", r.du, "u", dtype), ("ddelta", r.ddelta, "delta", dtype), ("dz", r.dz, "z", dtype),
                               ("dB", r.dB, "B", dtype), ("dC", r.dC, "C", dtype), ("dA", r.dA, "A", torch.float32),
                               ("dD", r.dD, "D", torch.float32), ("ddelta_bias", r.ddelta_bias, "bias", torch.float32)):
        R.check(got, gr[key], ty, TOL, name)
    if init:
        R.check(r.dinit, gr["st"], torch.float32, TOL, "dinit")


@pytest.mark.parametrize("use", [(), ("z",), ("D", "bias"), ("st",)], ids=str)
@pytest.mark.parametrize("softplus", [True, False])
def test_optional_inputs(use, softplus):
    t = make(2, 37, 96, 16, 1, torch.float32, seed=4)
    if not softplus:
        t["delta"] = t["delta"].abs() * 0.1
        t["bias"] = t["bias"].exp()
    g, t = on_gpu(t), views(t)
    pick = lambda k: g[k] if k in use else None
    y, f, kept = ssd.selective_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], pick("D"), pick("z"), pick("bias"),
                                   pick("st"), softplus=softplus, keep=True)
    r = ssd.selective_bwd(g["dy"], g["u"], g["delta"], g["A"], g["B"], g["C"], pick("D"), pick("z"), pick("bias"), kept,
                          softplus=softplus)
    torch.cuda.synchronize()
    t["df"] = torch.zeros_like(t["df"])
    yr, fr, gr = reference(t, use, softplus)
    R.check(y, yr, torch.float32, TOL, "y")
    R.check(f, fr, torch.float32, TOL, "final_state")
    for got, key in ((r.du, "u"), (r.ddelta, "delta"), (r.dA, "A"), (r.dB, "B"), (r.dC, "C"), (r.dD, "D"), (r.dz, "z"),
                     (r.ddelta_bias, "bias")):
        if got is None:
            assert key not in use
        else:
            R.check(got, gr[key], torch.float32, TOL, key)


@pytest.mark.parametrize("shape", [(600, 21, 128, 16, 1), (300, 11, 70, 32, 1), (9, 333, 520, 16, 2)], ids=str)
def test_one_chunk_and_many(shape):
    """Batches with waves enough for one pass, and long rows in many chunks."""
    b, L, d, N, G = shape
    t = make(b, L, d, N, G, torch.float32, seed=b, ragged=True)
    g = on_gpu(t)
    y, f, kept = ssd.selective_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], g["st"],
                                   lengths=g["lengths"], keep=True)
    r = ssd.selective_bwd(g["dy"], g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], kept,
                          dfinal=g["df"], lengths=g["lengths"])
    torch.cuda.synchronize()
    rows = [0, 1, b // 2, b - 1]
    sub = views({k: (v[rows].contiguous() if k in ("uz", "delta", "bc", "st", "dy", "df", "lengths") else v)
                 for k, v in t.items() if k not in ("u", "z", "B", "C")})
    yr, fr, gr = reference(sub, ("D", "z", "bias", "st"), True)
    R.check(y[rows], yr, torch.float32, TOL, "y")
    R.check(f[rows], fr, torch.float32, TOL, "final_state")
    for name, got, key in (("du", r.du, "u"), ("ddelta", r.ddelta, "delta"), ("dz", r.dz, "z"), ("dB", r.dB, "B"),
                           ("dC", r.dC, "C"), ("dinit", r.dinit, "st")):
        R.check(got[rows], gr[key], torch.float32, TOL, name)
    # what is summed over the batch: against the sum of one-row calls
    total = [torch.zeros_like(r.dA), torch.zeros_like(r.dD), torch.zeros_like(r.ddelta_bias)]
    for i in range(0, b, max(1, b // 8)):
        s = slice(i, min(b, i + max(1, b // 8)))
        a = [g["u"][s], g["delta"][s], g["A"], g["B"][s], g["C"][s], g["D"], g["z"][s], g["bias"]]
        _, _, k = ssd.selective_fwd(*a, g["st"][s], lengths=g["lengths"][s], keep=True)
        q = ssd.selective_bwd(g["dy"][s], *a, k, dfinal=g["df"][s], lengths=g["lengths"][s])
        for acc, v in zip(total, (q.dA, q.dD, q.ddelta_bias)):
            acc += v
    for got, ref, name in zip((r.dA, r.dD, r.ddelta_bias), total, ("dA", "dD", "ddelta_bias")):
        R.check(got, ref, torch.float32, TOL, name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,d,N,G", [(1, 1, 16, 1), (1, 1536, 16, 1), (5, 66, 32, 2), (33, 130, 64, 1), (3, 100, 16, 2)])
def test_steps_continue_a_prompt(b, d, N, G, dtype):
    L, T = 11, 4
    t = make(b, L + T, d, N, G, dtype, seed=d + N, extra=2)
    g, t = on_gpu(t), views(t)
    y, st = ssd.selective_fwd(*(g[k][:, :L] for k in ("u", "delta")), g["A"], g["B"][:, :L], g["C"][:, :L], g["D"],
                              g["z"][:, :L], g["bias"], g["st"])
    ys = []
    for k in range(L, L + T):
        out = torch.empty_like(st)
        a = (g["u"][:, k], g["delta"][:, k], g["A"], g["B"][:, k], g["C"][:, k], g["D"], g["z"][:, k], g["bias"], st)
        y2 = ssd.selective_step(*a, state_out=out)
        ys.append(ssd.selective_step(*a))
        assert torch.equal(st, out) and torch.equal(y2, ys[-1])
    torch.cuda.synchronize()
    yr, fr, _ = reference(t, ("D", "z", "bias", "st"), True, want=False)
    R.check(torch.cat([y, torch.stack(ys, 1)], 1), yr, dtype, TOL, "y")
    R.check(st, fr, torch.float32, TOL, "state")


def test_sequence_in_two_calls_and_in_place():
    """A sequence cut in two, the state carried in place, equals one call."""
    t = make(2, 300, 200, 16, 1, torch.float32, seed=8)
    g = on_gpu(t)
    args = lambda s: (g["u"][:, s], g["delta"][:, s], g["A"], g["B"][:, s], g["C"][:, s], g["D"], g["z"][:, s], g["bias"])
    y, f = ssd.selective_fwd(*args(slice(None)), g["st"])
    st = g["st"].clone()
    y1, f1 = ssd.selective_fwd(*args(slice(0, 123)), st, final_state=st)
    y2, f2 = ssd.selective_fwd(*args(slice(123, 300)), st, final_state=st)
    torch.cuda.synchronize()
    assert f1 is st and f2 is st
    R.check(torch.cat([y1, y2], 1), y, torch.float32, TOL, "y")
    R.check(st, f, torch.float32, TOL, "state")


def test_special_values():
    """A step size of zero keeps the state; a decay that underflows forgets it; a large step
    (softplus beyond its linear point) and a very negative one stay exact."""
    b, L, d, N = 1, 40, 64, 16
    t = make(b, L, d, N, 1, torch.float32, seed=2)
    t["bias"] = torch.zeros(d)
    t["delta"][:, :10] = -120.0              # dt underflows to 0: the state stays
    t["delta"][:, 10:20] = 50.0              # beyond the linear point: exp(-50 A) = 0
    t["delta"][:, 20:30] = -15.0             # log1p of 3e-7
    g, t = on_gpu(t), views(t)
    y, f, kept = ssd.selective_fwd(g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], g["st"], keep=True)
    r = ssd.selective_bwd(g["dy"], g["u"], g["delta"], g["A"], g["B"], g["C"], g["D"], g["z"], g["bias"], kept,
                          dfinal=g["df"])
    torch.cuda.synchronize()
    yr, fr, gr = reference(t, ("D", "z", "bias", "st"), True)
    R.check(y, yr, torch.float32, TOL, "y")
    R.check(y[:, :10], yr[:, :10], torch.float32, TOL, "y where dt = 0")
    R.check(f, fr, torch.float32, TOL, "final_state")
    for got, key in ((r.du, "u"), (r.ddelta, "delta"), (r.dA, "A"), (r.dB, "B"), (r.dC, "C"), (r.dz, "z"), (r.dinit, "st")):
        R.check(got, gr[key], torch.float32, TOL, key)


def test_gradient_against_differences():
    """Directional derivatives by central differences of the forward, in float32: truncation
    (4e-3)^2 and rounding 2e-6 / 4e-3 of the terms stay below 2e-3."""
    t = make(2, 60, 96, 16, 1, torch.float32, seed=6)
    g = on_gpu(t)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias")
    _, _, kept = ssd.selective_fwd(*(g[k] for k in keys), g["st"], keep=True)
    r = ssd.selective_bwd(g["dy"], *(g[k] for k in keys), kept, dfinal=g["df"])
    grads = dict(u=r.du, delta=r.ddelta, A=r.dA, B=r.dB, C=r.dC, D=r.dD, z=r.dz, bias=r.ddelta_bias, st=r.dinit)
    gen = torch.Generator().manual_seed(3)
    for key, grad in grads.items():
        v = torch.randn(g[key].shape, generator=gen).to(DEV)

        def loss(s):
            e = dict(g)
            e[key] = (g[key] + s * v)
            y, f = ssd.selective_fwd(*(e[k] for k in keys), e["st"])
            return float((y.double() * g["dy"].double()).sum() + (f.double() * g["df"].double()).sum())
        eps = 4e-3
        num, ana = (loss(eps) - loss(-eps)) / (2 * eps), float((grad.double() * v.double()).sum())
        size = float((grad.double().square().sum() * v.double().square().sum()).sqrt())
        assert abs(num - ana) <= 2e-3 * size, (key, num, ana, size)


def test_results_do_not_change_from_call_to_call():
    t = make(3, 200, 500, 16, 1, torch.bfloat16, seed=12, ragged=True)
    g = on_gpu(t)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias")
    first = None
    for k in range(3):
        y, f, kept = ssd.selective_fwd(*(g[k] for k in keys), g["st"], lengths=g["lengths"], keep=True)
        r = ssd.selective_bwd(g["dy"], *(g[k] for k in keys), kept, lengths=g["lengths"])
        torch.cuda.synchronize()
        now = (y, f) + tuple(r)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_nan_stays_in_its_channel():
    """A NaN step size or input reaches its own channel's later outputs and no other channel's."""
    t = make(1, 30, 130, 16, 1, torch.float32, seed=21)
    t["delta"][0, 10, 5] = float("nan")
    t["uz"][0, 12, 70] = float("nan")
    g = on_gpu(t)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias")
    y, f = ssd.selective_fwd(*(g[k] for k in keys), g["st"])
    clean = dict(g)
    clean["delta"], clean["uz"] = g["delta"].clone(), g["uz"].clone()
    clean["delta"][0, 10, 5], clean["uz"][0, 12, 70] = 0.0, 0.0
    clean = views(clean)
    yc, fc = ssd.selective_fwd(*(clean[k] for k in keys), g["st"])
    torch.cuda.synchronize()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 10:, 5], bad[0, 12:, 70] = True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], yc[~bad])
    assert torch.isnan(f[0, [5, 70]]).all() and torch.isfinite(f[0, [k for k in range(130) if k not in (5, 70)]]).all()


@pytest.mark.parametrize("L", [19, 24])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_last_token_s_input_reaches_no_earlier_gradient(L, bad):
    """The last token's u enters no state that a gradient of A or of an earlier token reads, in
    rows that end inside a group of 8 tokens too."""
    t = make(1, L, 130, 16, 1, torch.float32, seed=22)
    g = on_gpu(t)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias")
    out = []
    for value in (0.5, bad):
        e = dict(g)
        e["uz"] = g["uz"].clone()
        e["uz"][0, L - 1, 7] = value
        e = views(e)
        _, _, kept = ssd.selective_fwd(*(e[k] for k in keys), g["st"], keep=True)
        out.append(ssd.selective_bwd(g["dy"], *(e[k] for k in keys), kept))
    torch.cuda.synchronize()
    a, b = out
    assert torch.equal(a.dA, b.dA) and torch.equal(a.dinit, b.dinit)
    for name in ("du", "ddelta", "dz", "dB", "dC"):
        assert torch.equal(getattr(a, name)[:, :L - 1], getattr(b, name)[:, :L - 1]), name


def test_more_chunks_than_one_workgroup_holds_at_once():
    """5000 tokens of one tile: over 300 chunks, whose states pass through a workgroup in several
    rounds.  A state's memory reaches 1000 tokens here: 1000 * 4 * 2^-24 = 2.4e-4, doubled."""
    t = make(1, 5000, 64, 16, 1, torch.float32, seed=23)
    g, t = on_gpu(t), views(t)
    keys = ("u", "delta", "A", "B", "C", "D", "z", "bias")
    y, f, kept = ssd.selective_fwd(*(g[k] for k in keys), g["st"], keep=True)
    r = ssd.selective_bwd(g["dy"], *(g[k] for k in keys), kept, dfinal=g["df"])
    torch.cuda.synchronize()
    yr, fr, gr = reference(t, ("D", "z", "bias", "st"), True)
    R.check(y, yr, torch.float32, 5e-4, "y")
    R.check(f, fr, torch.float32, 5e-4, "final_state")
    for got, key in ((r.du, "u"), (r.ddelta, "delta"), (r.dz, "z"), (r.dB, "B"), (r.dC, "C"), (r.dA, "A"), (r.dD, "D"),
                     (r.ddelta_bias, "bias"), (r.dinit, "st")):
        R.check(got, gr[key], torch.float32, 5e-4, key)


def test_single_token_views_at_any_element():
    """A step takes B and C at any element's address."""
    t = make(3, 1, 96, 16, 1, torch.bfloat16, seed=24)
    g = on_gpu(t)
    odd = torch.zeros(3, 35, dtype=torch.bfloat16, device=DEV)
    odd[:, 1:33] = g["bc"][:, 0]
    a = (g["u"][:, 0], g["delta"][:, 0], g["A"])
    rest = (g["D"], g["z"][:, 0], g["bias"], g["st"])
    out, out2 = torch.empty_like(g["st"]), torch.empty_like(g["st"])
    y = ssd.selective_step(*a, g["B"][:, 0], g["C"][:, 0], *rest, state_out=out)
    y2 = ssd.selective_step(*a, odd[:, None, 1:17], odd[:, None, 17:33], *rest, state_out=out2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(out, out2)
