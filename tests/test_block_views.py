"""Inputs as views with strides of their own, and calls on another stream: the operators around
a scan give the bits that they give for contiguous tensors on the current stream."""
import pytest
import torch

from chunked_linear_recurrence_amd import ssd
from test_selective import make, on_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEYS = ("u", "delta", "A", "B", "C", "D", "z", "bias")


def wider(t, before, after, turned=False):
    """t as a view: channels `before` elements into rows wider by before + after; turned: tokens
    in front of the batch in memory."""
    shape = t.shape[:-1] + (before + t.shape[-1] + after,)
    if turned:
        full = torch.full((shape[1], shape[0], shape[2]), 7.0, dtype=t.dtype, device=t.device).transpose(0, 1)
    else:
        full = torch.full(shape, 7.0, dtype=t.dtype, device=t.device)
    v = full[..., before:before + t.shape[-1]]
    v.copy_(t)
    return v


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


VIEWS = [(8, 8, False), (3, 0, False), (1, 6, True), (0, 8, True)]       # on 16 bytes or off them


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("view", VIEWS, ids=str)
def test_convolution_backward_of_strided_gradients(view, dtype):
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(3, 37, 72, generator=gen).to(dtype).to(DEV) for _ in range(2))
    w, st = torch.randn(72, 4, generator=gen).to(DEV), torch.randn(3, 3, 72, generator=gen).to(dtype).to(DEV)
    ref = ssd.conv_bwd(dy, x, w, None, st)
    for a in (ssd.conv_bwd(wider(dy, *view), x, w, None, st), ssd.conv_bwd(dy, wider(x, *view), w, None, st),
              ssd.conv_bwd(wider(dy, *view), wider(x, *VIEWS[0]), w, None, st)):
        assert same(a, ref)
    broadcast = dy[:1, :1].expand(3, 37, 72)
    assert same(ssd.conv_bwd(broadcast, x, w, None, st), ssd.conv_bwd(broadcast.contiguous(), x, w, None, st))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("view", VIEWS[:2], ids=str)
def test_norm_of_strided_rows_and_gradients(view, dtype):
    gen = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(37, 72, generator=gen).to(dtype).to(DEV) for _ in range(2))
    w, b = torch.randn(72, generator=gen).to(DEV), torch.randn(72, generator=gen).to(DEV)
    y, mean, rstd = ssd.norm_fwd(x, w, b, want_stats=True)
    ref = ssd.norm_bwd(dy, x, w, mean, rstd)
    off = view[0] % 8 != 0          # other accesses, so the sums over a row are added in another order
    for dv, xv in ((wider(dy, *view), x), (dy, wider(x, *view)), (wider(dy, *view), wider(x, *view))):
        got = ssd.norm_bwd(dv, xv, w, mean, rstd)
        for p, q in zip(got, ref):
            if off:                 # 72 terms of 2^-24 each, and one rounding to storage
                bound = 72 * 2.0 ** -24 * float(q.float().abs().max()) + (2.0 ** -7 * q.float().abs() if p.dtype != torch.float32 else 0)
                assert ((p.float() - q.float()).abs() <= bound).all()
            else:
                assert torch.equal(p, q)
    assert off or torch.equal(ssd.norm_fwd(wider(x, *view), w, b), y)
    broadcast = dy[:1].expand(37, 72)
    assert same(ssd.norm_bwd(broadcast, x, w, mean, rstd), ssd.norm_bwd(broadcast.contiguous(), x, w, mean, rstd))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,G,L", [(16, 1, 70), (32, 2, 29)])
def test_scan_of_strided_inputs(N, G, L, dtype):
    """Each activation by itself and all of them together."""
    t = make(3, L, 130, N, G, dtype, seed=7, ragged=True)
    g = on_gpu(t)
    g = {k: (v.contiguous() if isinstance(v, torch.Tensor) else v) for k, v in g.items()}

    def call(e):
        y, f, kept = ssd.selective_fwd(*(e[k] for k in KEYS), e["st"], lengths=e["lengths"], keep=True)
        return (y, f) + tuple(ssd.selective_bwd(e["dy"], *(e[k] for k in KEYS), kept, dfinal=e["df"], lengths=e["lengths"]))
    ref = call(g)
    rows = lambda v, k: wider(v.flatten(-2), *k).unflatten(-1, v.shape[-2:]) if v.dim() == 4 else wider(v, *k)
    every = dict(g)
    for i, name in enumerate(("u", "delta", "z", "dy", "B", "C")):
        view = (2 * i, 2 * (i % 3), i % 2 == 1)                   # rows of B and C on 4 bytes
        every[name] = rows(g[name], view)
        assert same(call({**g, name: every[name]}), ref), name
    assert same(call(every), ref)
    for name in ("u", "delta", "z", "dy"):
        odd = wider(g[name], 1, 2)
        assert same(call({**g, name: odd}), ref), name
        one = g[name][:1, :1].expand_as(g[name])
        assert same(call({**g, name: one}), call({**g, name: one.contiguous()})), name


def test_calls_on_another_stream():
    """With stream=, every operator runs there: the current stream's work in front of it is waited
    for by the caller, and the results are the same bits."""
    t = make(2, 60, 96, 16, 1, torch.bfloat16, seed=9)
    g = on_gpu(t)
    x, w, st = g["u"].contiguous(), torch.randn(96, 4, device=DEV), torch.randn(2, 3, 96, device=DEV).bfloat16()
    nw = torch.randn(96, device=DEV)

    def calls(stream):
        y, f = ssd.conv_fwd(x, w, None, st, stream=stream)
        s = st.clone() if stream is None else clones[0]
        out = [y, f, ssd.conv_step(x[:, 0], w, None, s, stream=stream), s] + list(ssd.conv_bwd(g["dy"], x, w, None, st, stream=stream))
        y, f, kept = ssd.selective_fwd(*(g[k] for k in KEYS), g["st"], keep=True, stream=stream)
        h = g["st"].clone() if stream is None else clones[1]
        out += [y, f, ssd.selective_step(*(g[k][:, 0] if g[k].dim() > 2 else g[k] for k in KEYS), h, stream=stream), h]
        out += list(ssd.selective_bwd(g["dy"], *(g[k] for k in KEYS), kept, dfinal=g["df"], stream=stream))
        y, mean, rstd = ssd.norm_fwd(x.view(-1, 96), nw, nw, want_stats=True, stream=stream)
        out += [y, mean, rstd] + list(ssd.norm_bwd(g["dy"].view(-1, 96), x.view(-1, 96), nw, mean, rstd, stream=stream))
        return out
    ref = calls(None)
    side = torch.cuda.Stream()
    clones = (st.clone(), g["st"].clone())
    side.wait_stream(torch.cuda.current_stream())
    got = calls(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert same(got, ref)
