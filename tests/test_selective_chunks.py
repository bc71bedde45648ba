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
