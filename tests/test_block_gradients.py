"""Gradients through the block's operators in the combinations of optional inputs that the
operators take, against float64."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd import block, ssd

DEV = "cuda:0"


@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_norm_backward_returns_what_the_forward_was_given(weight, bias, monkeypatch):
    """Without a GPU, on values that stand for the kernels': autograd takes the gradients."""
    monkeypatch.setattr(ssd, "norm_fwd", lambda x, w, b, eps, want_stats: (x + 1, x[:, 0] * 0, x[:, 0] * 0))
    monkeypatch.setattr(ssd, "norm_bwd", lambda dy, x, w, m, r: ssd.NormGrads(dy + 0, dy.sum(0), dy.sum(0) * 2))
    x = torch.zeros(3, 4).requires_grad_(True)
    w = torch.ones(4).requires_grad_(True) if weight else None
    b = torch.ones(4).requires_grad_(True) if bias else None
    block.norm(x, w, b).sum().backward()
    assert torch.equal(x.grad, torch.ones(3, 4))
    assert w is None or torch.equal(w.grad, torch.full((4,), 3.0))
    assert b is None or torch.equal(b.grad, torch.full((4,), 6.0))


@pytest.mark.gpu
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_norm_with_and_without_parameters(weight, bias):
    """Tolerances of the norm's own tests: 2e-5 of the largest value, 1e-4 for sums over rows."""
    gen = torch.Generator().manual_seed(11)
    x, dy = torch.randn(37, 200, generator=gen) * 2 + 0.5, torch.randn(37, 200, generator=gen)
    w = 1 + 0.3 * torch.randn(200, generator=gen) if weight else None
    b = torch.randn(200, generator=gen) if bias else None
    leaves = [None if t is None else t.to(DEV).requires_grad_(True) for t in (x, w, b)]
    y = block.norm(*leaves)
    y.backward(dy.to(DEV))
    torch.cuda.synchronize()
    ref = [None if t is None else R.up(t).requires_grad_(True) for t in (x, w, b)]
    yr = R.norm(*ref)[0]
    grads = iter(R.grads((yr,), (R.up(dy),), [t for t in ref if t is not None]))
    R.check(y, yr, torch.float32, 2e-5, "y")
    for name, t, tol in zip(("x", "weight", "bias"), leaves, (2e-5, 1e-4, 1e-4)):
        if t is not None:
            R.check(t.grad, next(grads), torch.float32, tol, name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [float("nan"), float("inf")])
def test_what_lies_past_a_row_s_end_reaches_nothing(pad, dtype):
    """A ragged batch's padding may hold anything: outputs and states of the rows' own tokens and
    every gradient are those of a batch padded with zeros, bit for bit."""
    torch.manual_seed(8)
    m = block.SelectiveBlock(48, rank=4, dtype=dtype, device=DEV)
    lengths = torch.tensor([40, 0, 23], dtype=torch.int32, device=DEV)
    inside = torch.arange(40, device=DEV)[None] < lengths[:, None]
    x, dy = torch.randn(3, 40, 48, device=DEV).to(dtype), torch.randn(3, 40, 48, device=DEV).to(dtype)
    dy[~inside] = 0
    got = []
    for value in (0.0, pad):
        xp = x.clone()
        xp[~inside] = value
        xp.requires_grad_(True)
        m.zero_grad()
        y, state = m(xp, lengths=lengths)
        y.backward(dy)
        got.append([y[inside], *state, xp.grad] + [p.grad.clone() for p in m.parameters()])
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.isfinite(b).all() and torch.equal(a, b)
