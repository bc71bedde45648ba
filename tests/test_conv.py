"""The short causal convolution (conv_fwd, conv_step, conv_bwd) against float64.

Tolerance: a result is W + 1 products and sums of float32 (each 2^-24), a SiLU of a few ulp
and its own rounding; the terms of a sum may exceed the sum's largest value a few times.
20 * 2^-24 times a factor of 8 is below 1e-5 of the largest value.  Sums over tokens (weight
and bias gradients) add at most 64 * 2^-24 in a running sum per wave and partial sums in
sequence: 1e-4 covers them."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL, TOL_SUM = 1e-5, 1e-4


def make(b, L, C, W, dtype, seed, split=False, init=True, ragged=False, pad=None):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(b, L, 2 * C if split else C, generator=g).to(dtype)
    x = full[..., :C] if not split else full[..., C:]
    w = torch.randn(C, W, generator=g) / W ** 0.5
    bias = torch.randn(C, generator=g) * 0.2
    st = torch.randn(b, W - 1, C, generator=g).to(dtype) if init else None
    lengths = None
    if ragged:
        lengths = torch.randint(0, L + 1, (b,), generator=g, dtype=torch.int32)
        lengths[0], lengths[-1] = L, 0
    dy = torch.randn(b, L, C, generator=g).to(dtype)
    if ragged and pad is not None:
        for i in range(b):
            x[i, int(lengths[i]):] = pad
            dy[i, int(lengths[i]):] = pad
    df = torch.randn(b, W - 1, C, generator=g).to(dtype)
    return dict(full=full, x=x, w=w, bias=bias, st=st, lengths=lengths, dy=dy, df=df)


def on_gpu(t, split):
    d = {k: (v.to(DEV) if v is not None else None) for k, v in t.items()}
    C = t["x"].shape[2]
    d["x"] = d["full"][..., C:] if split else d["full"]
    return d


SHAPES = [  # b, L, C, W, split, init, ragged
    (1, 1, 1, 2, False, False, False), (1, 1, 64, 4, False, True, False), (2, 2, 65, 4, False, True, False),
    (3, 3, 8, 4, False, True, True), (2, 15, 72, 3, True, True, True), (1, 16, 512, 4, False, False, False),
    (2, 17, 520, 4, True, True, False), (4, 63, 7, 2, False, True, True), (2, 64, 1032, 3, False, True, True),
    (3, 65, 96, 4, True, False, True), (2, 129, 777, 4, False, True, True), (1, 1000, 40, 4, False, True, False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("silu", [True, False])
def test_forward_and_backward(shape, dtype, silu):
    b, L, C, W, split, init, ragged = shape
    t = make(b, L, C, W, dtype, seed=L * C + W, split=split, init=init, ragged=ragged,
             pad=float("nan") if L % 2 else float("inf"))
    d = on_gpu(t, split)
    bias = t["bias"] if C % 3 else None
    dbias = None if bias is None else d["bias"]
    y, fin = ssd.conv_fwd(d["x"], d["w"], dbias, d["st"], lengths=d["lengths"], silu=silu)
    g = ssd.conv_bwd(d["dy"], d["x"], d["w"], dbias, d["st"], dfinal=d["df"], lengths=d["lengths"], silu=silu)
    torch.cuda.synchronize()
    x, w, st = R.up(t["x"]), R.up(t["w"]), R.up(t["st"])
    rb = R.up(bias)
    leaves = [v.requires_grad_(True) for v in (x, w, rb, st) if v is not None]
    yr, fr = R.conv(x, w, rb, st, t["lengths"], silu)
    gr = dict(zip([n for n, v in (("dx", x), ("dweight", w), ("dbias", rb), ("dinit", st)) if v is not None],
                  R.grads((yr, fr), (R.up(t["dy"]), R.up(t["df"])), leaves)))
    R.check(y, yr, dtype, TOL, "y")
    R.check(fin, fr, dtype, 0.0, "final_state")
    R.check(g.dx, gr["dx"], dtype, TOL, "dx")
    R.check(g.dweight, gr["dweight"], torch.float32, TOL_SUM, "dweight")
    if bias is not None:
        R.check(g.dbias, gr["dbias"], torch.float32, TOL_SUM, "dbias")
    else:
        assert g.dbias is None
    if init:
        R.check(g.dinit, gr["dinit"], dtype, TOL, "dinit")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,C,W", [(1, 1, 2), (1, 1536, 4), (7, 65, 3), (33, 264, 4)])
def test_steps_continue_a_prompt(b, C, W, dtype):
    """A prompt and then single tokens, in place, equal the whole sequence; state_out leaves
    the incoming state alone."""
    L, T = 9, 5
    t = make(b, L + T, C, W, dtype, seed=C, init=True)
    d = on_gpu(t, False)
    y, st = ssd.conv_fwd(d["x"][:, :L], d["w"], d["bias"], d["st"])
    ys = []
    for k in range(T):
        before = st.clone()
        out = torch.empty_like(st)
        y2 = ssd.conv_step(d["x"][:, L + k], d["w"], d["bias"], st, state_out=out)
        assert torch.equal(st, before)
        ys.append(ssd.conv_step(d["x"][:, L + k], d["w"], d["bias"], st))
        assert torch.equal(st, out) and torch.equal(ys[-1], y2)
    torch.cuda.synchronize()
    yr, fr = R.conv(R.up(t["x"]), R.up(t["w"]), R.up(t["bias"]), R.up(t["st"]))
    R.check(torch.cat([y, torch.stack(ys, 1)], 1), yr, dtype, TOL, "y")
    R.check(st, fr, dtype, 0.0, "state")


@pytest.mark.parametrize("L", [1, 2, 5, 40])
def test_state_in_place_and_other_stream(L):
    """final_state may be init_state, also for rows shorter than the state; a call on another
    stream gives the same bits."""
    t = make(3, L, 136, 4, torch.bfloat16, seed=L, ragged=True)
    d = on_gpu(t, False)
    y, fin = ssd.conv_fwd(d["x"], d["w"], d["bias"], d["st"], lengths=d["lengths"])
    st = d["st"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, fin2 = ssd.conv_fwd(d["x"], d["w"], d["bias"], st, lengths=d["lengths"], final_state=st, stream=side)
    torch.cuda.synchronize()
    assert fin2 is st and torch.equal(st, fin) and torch.equal(y, y2)


def test_misaligned_views_give_the_same_bits():
    """Rows that start off a 16-byte boundary take element accesses; the arithmetic is the same."""
    t = make(2, 50, 64, 4, torch.bfloat16, seed=1)
    d = on_gpu(t, False)
    odd = torch.zeros(2, 50, 67, dtype=torch.bfloat16, device=DEV)
    odd[..., 3:] = d["x"]
    y, f = ssd.conv_fwd(d["x"], d["w"], d["bias"], d["st"])
    y2, f2 = ssd.conv_fwd(odd[..., 3:], d["w"], d["bias"], d["st"])
    g = ssd.conv_bwd(d["dy"], d["x"], d["w"], d["bias"], d["st"])
    g2 = ssd.conv_bwd(d["dy"], odd[..., 3:], d["w"], d["bias"], d["st"])
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(f, f2)
    for a, b in zip(g, g2):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """The change of a loss along a random direction, by central differences of the forward:
    truncation (1e-2)^2 and rounding 1e-6 / 1e-2 of the loss's terms stay below 1e-3."""
    t = make(2, 40, 70, 4, torch.float32, seed=5)
    d = on_gpu(t, False)
    g = ssd.conv_bwd(d["dy"], d["x"], d["w"], d["bias"], d["st"], dfinal=d["df"])
    gen = torch.Generator().manual_seed(9)
    for name, grad, key in (("x", g.dx, "x"), ("w", g.dweight, "w"), ("bias", g.dbias, "bias"), ("st", g.dinit, "st")):
        v = torch.randn(d[key].shape, generator=gen).to(DEV)

        def loss(s):
            e = dict(d)
            e[key] = d[key] + s * v
            y, f = ssd.conv_fwd(e["x"], e["w"], e["bias"], e["st"])
            return float((y.double() * d["dy"].double()).sum() + (f.double() * d["df"].double()).sum())
        eps = 1e-2
        num, ana = (loss(eps) - loss(-eps)) / (2 * eps), float((grad.double() * v.double()).sum())
        size = float((grad.double().square().sum() * v.double().square().sum()).sqrt())
        assert abs(num - ana) <= 1e-3 * size, (name, num, ana, size)
