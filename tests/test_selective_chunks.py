"""The selective scan's cut of a sequence into chunks: what a call gives must not depend on it.
Against float64; the tolerance is the scan's own (2e-4 of the largest value: 4 roundings a token
over the tokens that a state lives)."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd
from test_selective import TOL, make, on_gpu, reference, views

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEYS = ("u", "delta", "A", "B", "C", "D", "z", "bias")
GRADS = (("du", "u"), ("ddelta", "delta"), ("dz", "z"), ("dB", "B"), ("dC", "C"), ("dA", "A"), ("dD", "D"),
         ("ddelta_bias", "bias"), ("dinit", "st"))


@pytest.mark.parametrize("rate,L", [(0.6, 700), (0.6, 2000), (6.0, 100), (6.0, 700)], ids=str)
def test_growing_states_from_and_to_nothing(rate, L):
    """Decays above 1, finite for every token, whose product over a chunk or over the chunks of a
    wave is not: a state (a carry, backwards) of zero stays zero through them.  Inputs in the last
    10 tokens and upstream gradients in the first 10 alone, so that no result overflows (e^60)."""
    t = make(1, L, 70, 16, 1, torch.float32, seed=31, init=False)
    t["A"] = t["A"].abs().clamp(max=1.0) * 0 + rate
    t["delta"][:] = 1.0
    t["uz"][:, :-10, :70] = 0
    t["dy"][:, 10:] = 0
    t["df"].zero_()
    t["bias"].zero_()
    g, t = on_gpu(t), views(t)
    y, f, kept = ssd.selective_fwd(*(g[k] for k in KEYS), softplus=False, keep=True)
    r = ssd.selective_bwd(g["dy"], *(g[k] for k in KEYS), kept, softplus=False)
    torch.cuda.synchronize()
    assert ssd.lib().ssd_selective_fwd_workspace_bytes(ssd._selective_inputs(*(g[k] for k in KEYS), False)[0]) > 0
    yr, fr, gr = reference(t, ("D", "z", "bias"), False)
    R.check(y, yr, torch.float32, TOL, "y")
    R.check(f, fr, torch.float32, TOL, "final_state")
    for name, key in GRADS[:-1]:
        R.check(getattr(r, name), gr[key], torch.float32, TOL, name)


def test_growth_beyond_float32_s_range_of_a_small_state():
    """A chunk's product of decays may exceed float32 (e^96) where the state it acts on is small
    (1e-30): the state after it is finite."""
    L = 64
    t = make(1, L, 70, 16, 1, torch.float32, seed=32)
    t["A"] = torch.ones_like(t["A"])
    t["st"] = t["st"].sign() * 1e-30
    t["uz"][..., :70] = 0
    t["delta"][:] = 0
    t["delta"][:, :16] = 6.0
    t["bias"].zero_()
    g, t = on_gpu(t), views(t)
    y, f = ssd.selective_fwd(*(g[k] for k in KEYS), g["st"], softplus=False)
    torch.cuda.synchronize()
    yr, fr, _ = reference(t, ("D", "z", "bias", "st"), False, want=False)
    R.check(f, fr, torch.float32, TOL, "final_state")
    R.check(y, yr, torch.float32, TOL, "y")


# ---- which way a sequence is cut: one pass by its waves, and chunks longer than the shortest
def chunks(b, L, d, N, G, dims):
    """Chunks of the forward's cut, from the workspace it asks for (0: one pass)."""
    tiles = G * -(-(d // G) // 64)
    return ssd.lib().ssd_selective_fwd_workspace_bytes(dims) // (b * tiles * 64 * 4 * (N + 1))


def backward_in_one_pass(b, L, d, N, G, dims):
    """Whether the backward's workspace is that of its partial sums alone."""
    up = lambda v: -(-v // 256) * 256
    tiles = -(-(d // G) // 64)
    parts = -(-tiles // (64 // N))
    return ssd.lib().ssd_selective_bwd_workspace_bytes(dims) == (
        up(parts * b * L * G * 2 * N * 4) + up(b * G * tiles * 64 * 4 * (N + 2)))


def check_sampled_rows(shape, dtype, one_pass):
    """Every output and gradient against float64.  Upstream gradients are zero in all rows but
    four, which then give the whole of dA, dD and ddelta_bias.  delta and dy are views into wider
    rows, each with strides of its own."""
    b, L, d, N, G = shape
    t = make(b, L, d, N, G, dtype, seed=b + L, ragged=True, pad=float("nan"), extra=2)
    rows = [0, 1, b // 2, b - 1]
    t["lengths"][b // 2] = L - 5
    other = [i for i in range(b) if i not in rows]
    t["dy"][other], t["df"][other] = 0, 0
    for i in rows:
        t["dy"][i] = torch.randn(L, d, generator=torch.Generator().manual_seed(i)).to(dtype)
        t["delta"][i] = torch.nan_to_num(t["delta"][i], nan=0.25)
        t["uz"][i], t["bc"][i] = torch.nan_to_num(t["uz"][i], nan=0.5), torch.nan_to_num(t["bc"][i], nan=0.5)
    g = on_gpu(t)
    for key, extra in (("delta", 6), ("dy", 10)):
        wide = torch.zeros(b, L, d + extra, dtype=dtype, device=DEV)
        wide[..., extra // 2:extra // 2 + d] = g[key]
        g[key] = wide[..., extra // 2:extra // 2 + d]
    dims = ssd._selective_inputs(*(g[k] for k in KEYS), False, g["dy"])[0]
    n = chunks(b, L, d, N, G, dims)
    if one_pass:
        assert n == 0 and L > 32 and backward_in_one_pass(b, L, d, N, G, dims)
    else:
        assert n > 1 and n * 16 < L and not backward_in_one_pass(b, L, d, N, G, dims)
    y, f, kept = ssd.selective_fwd(*(g[k] for k in KEYS), g["st"], lengths=g["lengths"], keep=True)
    r = ssd.selective_bwd(g["dy"], *(g[k] for k in KEYS), kept, dfinal=g["df"], lengths=g["lengths"])
    torch.cuda.synchronize()
    sub = {k: (v[rows].contiguous() if k in ("uz", "delta", "bc", "st", "dy", "df", "lengths") else v)
           for k, v in t.items() if k not in ("u", "z", "B", "C")}
    yr, fr, gr = reference(views(sub), ("D", "z", "bias", "st"), True)
    R.check(y[rows], yr, dtype, TOL, "y")
    R.check(f[rows], fr, torch.float32, TOL, "final_state")
    for name, key in GRADS:
        got = getattr(r, name)
        whole = name in ("dA", "dD", "ddelta_bias")
        R.check(got if whole else got[rows], gr[key], torch.float32 if whole or name == "dinit" else dtype, TOL, name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(800, 57, 128, 16, 1), (790, 45, 130, 32, 2), (520, 70, 192, 64, 1)], ids=str)
def test_one_pass_by_the_number_of_waves(shape, dtype):
    check_sampled_rows(shape, dtype, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(30, 450, 1600, 16, 2), (40, 500, 1110, 32, 2), (44, 400, 640, 64, 1)], ids=str)
def test_chunks_longer_than_the_shortest(shape, dtype):
    check_sampled_rows(shape, dtype, False)
