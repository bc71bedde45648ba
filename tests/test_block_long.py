"""Tensors beyond 2^31 elements, and lengths outside a row: the operators around a scan."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_offsets_beyond_31_bits():
    """One row of 2^20 tokens and 2112 channels (2.2e9 elements): the end of the sequence, run again
    from the states that enter it, gives the same outputs and gradients (float32 operators' own
    tolerances; bfloat16 storage)."""
    L, d, N, T = 1 << 20, 2112, 16, 1000
    assert L * d > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(0)
    cut = L - T
    x = torch.randn(1, L, d, generator=g, device=DEV, dtype=torch.bfloat16)
    w, bias = torch.randn(d, 4, generator=g, device=DEV) * 0.5, torch.randn(d, generator=g, device=DEV)
    u, last = ssd.conv_fwd(x, w, bias)
    tail, last2 = ssd.conv_fwd(x[:, cut:], w, bias, x[:, cut - 3:cut].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(u[:, cut:], tail) and torch.equal(last, last2)
    gr = ssd.conv_bwd(x, x, w, bias)
    gt = ssd.conv_bwd(x[:, cut:], x[:, cut:], w, bias, x[:, cut - 3:cut].contiguous())
    assert torch.equal(gr.dx[:, cut:], gt.dx)
    del gr, gt, tail
    y = ssd.norm_fwd(u[0])
    assert torch.equal(y[cut:], ssd.norm_fwd(u[0, cut:].contiguous()))
    del y
    delta = torch.randn(1, L, d, generator=g, device=DEV, dtype=torch.bfloat16).mul_(0.5)
    A = -torch.rand(d, N, generator=g, device=DEV) * 16 - 0.5
    B = torch.randn(1, L, 1, N, generator=g, device=DEV, dtype=torch.bfloat16)
    C = torch.randn(1, L, 1, N, generator=g, device=DEV, dtype=torch.bfloat16)
    D, db = torch.rand(d, generator=g, device=DEV), torch.full((d,), -3.0, device=DEV)
    args = lambda s: (u[:, s], delta[:, s], A, B[:, s], C[:, s], D, x[:, s], db)
    y, end, kept = ssd.selective_fwd(*args(slice(None)), keep=True)
    _, mid = ssd.selective_fwd(*args(slice(0, cut)))
    y2, end2, kept2 = ssd.selective_fwd(*args(slice(cut, L)), mid, keep=True)
    R.check(y[:, cut:], y2, torch.bfloat16, 2e-4, "y")
    R.check(end, end2, torch.float32, 2e-4, "state")
    gr = ssd.selective_bwd(u, *args(slice(None)), kept)
    gt = ssd.selective_bwd(u[:, cut:], *args(slice(cut, L)), kept2)
    torch.cuda.synchronize()
    for name in ("du", "ddelta", "dz", "dB", "dC"):
        R.check(getattr(gr, name)[:, cut:], getattr(gt, name), torch.bfloat16, 2e-4, name)
    # the first tokens' gradients, against a run over a prefix whose memory ends well inside it
    # (decays of at least exp(-0.5 * softplus(-4)) a token over 2000 tokens)
    head = ssd.selective_fwd(*args(slice(0, 4000)), keep=True)
    gh = ssd.selective_bwd(u[:, :4000], *args(slice(0, 4000)), head[2])
    for name in ("du", "ddelta", "dz", "dB", "dC"):
        R.check(getattr(gr, name)[:, :2000], getattr(gh, name)[:, :2000], torch.bfloat16, 2e-4, name)


def test_lengths_outside_a_row_are_clamped():
    """Negative lengths are 0 and lengths beyond the tokens are all of them."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 20, 64, generator=g).to(DEV)
    w, st = torch.randn(64, 4, generator=g).to(DEV), torch.randn(3, 3, 64, generator=g).to(DEV)
    odd = torch.tensor([-5, 1 << 30, 7], dtype=torch.int32, device=DEV)
    even = torch.tensor([0, 20, 7], dtype=torch.int32, device=DEV)
    for a, b in zip(ssd.conv_fwd(x, w, None, st, lengths=odd), ssd.conv_fwd(x, w, None, st, lengths=even)):
        assert torch.equal(a, b)
    for a, b in zip(ssd.conv_bwd(x, x, w, None, st, lengths=odd), ssd.conv_bwd(x, x, w, None, st, lengths=even)):
        assert (a is None and b is None) or torch.equal(a, b)
    A = -torch.rand(64, 16, generator=g).to(DEV)
    B = torch.randn(3, 20, 1, 16, generator=g).to(DEV)
    h = torch.randn(3, 64, 16, generator=g).to(DEV)
    outs = []
    for lengths in (odd, even):
        y, f, kept = ssd.selective_fwd(x, x, A, B, B, None, x, None, h, lengths=lengths, keep=True)
        outs.append([y, f] + [t for t in ssd.selective_bwd(x, x, x, A, B, B, None, x, None, kept, lengths=lengths)
                              if t is not None])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert float(outs[0][0][0].abs().max()) == 0.0 and torch.equal(outs[0][1][0], h[0])
