"""The operators of a layer's feed-forward half together: a layer's gradients against float64, a
ragged prompt and its continuation token by token, a training step with clipping, calls on other
streams and in graphs, and the functions with each combination of inputs."""
import itertools

import pytest
import torch

import block_ref as R
import ffn_ref
from chunked_linear_recurrence_amd import block as B
from chunked_linear_recurrence_amd import ssd
from test_block import reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rms(v):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)


def layer_reference(layer, x, lengths):
    """The layer in float64 on the CPU; (y, state) and its leaves."""
    if lengths is not None:
        keep = torch.arange(x.shape[1])[None, :] < torch.tensor([int(v) for v in lengths])[:, None]
        x = x * keep[..., None]
    out, state, p = reference(layer.block, x, None, lengths)
    p = {"block." + k: v for k, v in p.items()}
    q = {k: R.up(v).requires_grad_(True) for k, v in layer.named_parameters(recurse=False)}
    total = x + q["scale"] * (out - x)
    g, u = (rms(total) * q["norm_weight"] @ q["in_proj"].t()).chunk(2, -1)
    y = total + (ffn_ref.act(g, layer.act) * u) @ q["out_proj"].t()
    return y, state, {**q, **p}


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_through_a_layer(ragged, act):
    """float32; tolerance: the block's (4e-4 of the largest value), again through two products and
    a norm of it."""
    torch.manual_seed(3)
    layer = B.SelectiveLayer(48, 100, act=act, dstate=16, rank=4, dtype=torch.float32, device=DEV)
    x, dy = torch.randn(3, 70, 48), torch.randn(3, 70, 48)
    lengths = torch.tensor([70, 0, 33], dtype=torch.int32) if ragged else None
    xg = x.to(DEV)
    if ragged:                           # what lies behind a row's own tokens reaches nothing
        for i, m in enumerate(lengths.tolist()):
            xg[i, m:] = float("nan")
    xg.requires_grad_(True)
    y, state = layer(xg, lengths=None if lengths is None else lengths.to(DEV))
    (y * dy.to(DEV)).sum().backward()
    torch.cuda.synchronize()
    xr = R.up(x).requires_grad_(True)
    yr, sr, p = layer_reference(layer, xr, lengths)
    grads = R.grads((yr,), (R.up(dy),), [xr] + list(p.values()))
    R.check(y, yr, torch.float32, 8e-4, "y")
    R.check(state[1], sr[1], torch.float32, 4e-4, "scan state")
    R.check(xg.grad, grads[0], torch.float32, 8e-4, "x")
    mine = dict(layer.named_parameters())
    for name, g in zip(p, grads[1:]):
        R.check(mine[name].grad, g, torch.float32, 8e-4, name)


def test_prompt_then_tokens():
    """bfloat16: the same roundings in both, so the prompt's outputs and the steps' differ by the
    products' order of addition, and where that moves a rounding; 2e-2 of the largest value, as
    for the block."""
    torch.manual_seed(4)
    layer = B.SelectiveLayer(96, device=DEV)
    x = torch.randn(5, 60, 96, device=DEV).bfloat16()
    with torch.no_grad():
        whole, _ = layer(x)
        y, state = layer(x[:, :41].contiguous())
        ys = [layer.step(x[:, t], state) for t in range(41, 60)]
    got = torch.cat([y, torch.stack(ys, 1)], 1)
    assert float((got.float() - whole.float()).abs().max()) <= 2e-2 * float(whole.float().abs().max())


def test_training_step_clips():
    """A layer's gradients, clipped, have the norm asked for, and the same directions."""
    torch.manual_seed(5)
    layer = B.SelectiveLayer(64, device=DEV)
    y, _ = layer(torch.randn(2, 30, 64, device=DEV).bfloat16())
    y.float().square().sum().backward()
    grads = [p.grad for p in layer.parameters()]
    before = [g.clone() for g in grads]
    norm = ssd.clip_grads(grads, 1.0)
    ref = float(torch.sqrt(sum(g.double().square().sum() for g in before)))
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref and ref > 1.0
    # each value rounded once, by half a step at most: the sum of squares by twice 2^-8
    assert abs(float(ssd.grad_norm(grads)) - 1.0) <= 2.0 ** -7
    for a, b in zip(before, grads):
        assert ((b.double() - a.double() / ref).abs() <= 2.0 ** -7 * (a.double() / ref).abs() + 1e-38).all()


def test_decode_step_in_a_graph():
    """The single-token path captured and replayed, with eager work between the replays, gives
    the eager results bit for bit."""
    torch.manual_seed(6)
    layer = B.SelectiveLayer(64, device=DEV)
    x = torch.randn(3, 64, device=DEV).bfloat16()
    with torch.no_grad():
        _, first = layer(torch.randn(3, 9, 64, device=DEV).bfloat16())
    state = tuple(t.clone() for t in first)
    ref = [layer.step(x, state).clone() for _ in range(3)]
    static = tuple(t.clone() for t in first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x, static)
    for t, f in zip(static, first):
        t.copy_(f)
    for k in range(3):
        torch.randn(100, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[k]), k


def calls(seed):
    """Every operator once, forwards and backwards, in sizes that take each way through them:
    few rows, tiles of each size, K cut, operands laid out anew."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen, device=DEV).to(dt)
    data = []
    for m, k, n, dt in ((3, 200, 136, torch.bfloat16), (100, 4096, 64, torch.bfloat16), (700, 1001, 903, torch.bfloat16),
                        (2901, 136, 2840, torch.bfloat16), (300, 333, 200, torch.float32)):
        data.append((r(m, k, dt=dt), r(n, k, dt=dt), r(n, dt=dt), r(m, n, dt=dt)))
    norm = [(r(m, d), r(m, d), r(m, d), r(d, dt=torch.float32), r(d, dt=torch.float32), r(d, dt=torch.float32))
            for m, d in ((50, 512), (9, 9000))]
    grads = [r(5000), r(77, dt=torch.float32), r(3)]
    outs = [torch.empty_like(g) for g in grads]

    def run():
        got = []
        for x, w, b, y in data:
            o, pre = ssd.linear_fwd(x, w, b, y, act="silu", keep=True)
            got += [o, *ssd.linear_bwd(y, x, w, b, pre, act="silu")]
            if w.shape[0] % 2 == 0:
                f = w.shape[0] // 2
                h, pre = ssd.gated_fwd(x, w, b, act="gelu", keep=True)
                got += [h, *ssd.gated_bwd(y[:, :f], x, w, b, pre, act="gelu")]
        for br, re, z, post, sc, pre in norm:
            y, total, stats = ssd.residual_norm_fwd(br, re, z, post, sc, pre, want_stats=True)
            got += [y, total, *ssd.residual_norm_bwd(re, z, br, re, z, post, sc, pre, stats)]
        got += [ssd.clip_grads(grads, 1.0, out=outs), ssd.grad_norm(grads), *outs]
        return got
    return run, [t for group in data + norm for t in group] + grads


def test_on_another_stream():
    """Given as an argument or as the current one, with the default stream busy."""
    run, _ = calls(1)
    ref = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device=DEV)
    for _ in range(5):
        a = a @ a * 1e-4
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    x, w = torch.randn(300, 256, device=DEV).bfloat16(), torch.randn(128, 256, device=DEV).bfloat16()
    torch.cuda.synchronize()
    y = ssd.linear_fwd(x, w, stream=side)
    g = ssd.linear_bwd(y, x, w, stream=side)
    h, pre = ssd.gated_fwd(x, w, keep=True, stream=side)
    gg = ssd.gated_bwd(h, x, w, None, pre, stream=side)
    n, total, st = ssd.residual_norm_fwd(x, pre_weight=torch.ones(256, device=DEV), want_stats=True, stream=side)
    gn = ssd.residual_norm_bwd(n, None, x, None, None, None, None, torch.ones(256, device=DEV), st, stream=side)
    c = ssd.grad_norm([x, w], stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    y2 = ssd.linear_fwd(x, w)
    h2, pre2 = ssd.gated_fwd(x, w, keep=True)
    assert torch.equal(y, y2) and torch.equal(g.dx, ssd.linear_bwd(y2, x, w).dx)
    assert torch.equal(h, h2) and torch.equal(gg.dweight, ssd.gated_bwd(h2, x, w, None, pre2).dweight)
    assert torch.equal(n, ssd.residual_norm_fwd(x, pre_weight=torch.ones(256, device=DEV))[0]) and torch.isfinite(gn.dbranch).all()
    assert torch.equal(c, ssd.grad_norm([x, w]))


def test_captured_and_replayed():
    """Everything in one graph, and a second graph of other data whose workspaces may lie where the
    first's lie; replays with new inputs and eager work between them equal eager calls."""
    graphs = []
    pool = None
    for seed in (2, 3):
        run, inputs = calls(seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = run()
        pool = pool or graph.pool()
        graphs.append((graph, run, inputs, out))
    for k in range(3):
        for graph, run, inputs, out in graphs:
            for t in inputs:
                t.copy_(torch.randn_like(t.float()))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            ref = run()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(ref, got)), k


def test_two_calls_at_once():
    """The same operators on two streams at the same time do not meet."""
    runs = [calls(s) for s in (4, 5)]
    refs = [[t.clone() for t in run()] for run, _ in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = []
        for s, (run, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(refs, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("given", list(itertools.product([False, True], repeat=2)), ids=str)
def test_linear_function(given):
    """Gradients of each input alone, and of those that need none not at all."""
    bias, residual = given
    gen = torch.Generator().manual_seed(8)
    t = [torch.randn(*s, generator=gen) for s in ((40, 24), (56, 24), (56,), (40, 56))]
    ins = [t[0], t[1], t[2] if bias else None, t[3] if residual else None]
    dy = torch.randn(40, 56, generator=gen)
    for wanted in range(4):
        if ins[wanted] is None:
            continue
        a = [None if v is None else v.to(DEV).requires_grad_(i == wanted) for i, v in enumerate(ins)]
        B.linear(*a, act="gelu").backward(dy.to(DEV))
        r = [None if v is None else R.up(v).requires_grad_(i == wanted) for i, v in enumerate(ins)]
        y = ffn_ref.act(r[0] @ r[1].t() + (0 if r[2] is None else r[2]), "gelu") + (0 if r[3] is None else r[3])
        y.backward(R.up(dy))
        R.check(a[wanted].grad, r[wanted].grad, torch.float32, 1e-5, "gradient %d" % wanted)
        assert all(v is None or v.grad is None for i, v in enumerate(a) if i != wanted)


def test_broadcast_and_transposed_gradients():
    """A gradient that is one value for all (a sum's), and one whose columns do not lie together."""
    x, w = torch.randn(30, 16, device=DEV).requires_grad_(True), torch.randn(24, 16, device=DEV).requires_grad_(True)
    B.linear(x, w).sum().backward()
    torch.testing.assert_close(x.grad, w.detach().sum(0).expand(30, -1), rtol=1e-5, atol=1e-5)
    x.grad = w.grad = None
    g = torch.randn(12, 30, device=DEV)
    B.gated(x, w).t().backward(g)
    xr, wr = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    a, u = (xr @ wr.t()).chunk(2, 1)
    (torch.nn.functional.silu(a) * u).t().backward(g.double())
    torch.testing.assert_close(x.grad.double(), xr.grad, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(w.grad.double(), wr.grad, rtol=1e-4, atol=1e-4)
    b = torch.randn(5, 8, device=DEV).requires_grad_(True)
    y, total = B.residual_norm(b, pre_weight=torch.ones(8, device=DEV))
    total.sum().backward()                             # y unused
    assert torch.equal(b.grad, torch.ones_like(b))


def test_second_derivatives_and_stale_inputs_are_refused():
    x, w = torch.randn(6, 8, device=DEV).requires_grad_(True), torch.randn(4, 8, device=DEV)
    for f in (lambda v: B.linear(v, w), lambda v: B.gated(v, w), lambda v: B.residual_norm(v, pre_weight=torch.ones(8, device=DEV))[0]):
        (dx,) = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            dx.sum().backward()
    r = torch.randn(6, 8, device=DEV)
    y, _ = B.residual_norm(x, r, pre_weight=torch.ones(8, device=DEV))
    ssd.residual_norm_fwd(r.clone(), r, total=r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
