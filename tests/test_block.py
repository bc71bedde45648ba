"""The operators together, as a block uses them: views of projections, gradients through all of
them, a ragged prompt and its continuation token by token, against float64."""
import pytest
import torch

import block_ref as R
from chunked_linear_recurrence_amd.block import SelectiveBlock

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(block, x, state, lengths):
    """The block in float64 on the CPU from its definition; (y, state) and its leaves."""
    p = {k: R.up(v).requires_grad_(True) for k, v in block.named_parameters()}
    d, n, r = block.channels, block.dstate, block.rank
    b, L, w = x.shape
    h = R.norm(x.reshape(b * L, w), p["norm_weight"], p["norm_bias"])[0]
    xz = (h @ p["in_proj"].t()).view(b, L, 2 * d)
    u, cs = R.conv(xz[..., :d], p["conv_weight"], p["conv_bias"], None if state is None else state[0], lengths)
    q = u @ p["x_proj"].t()
    delta = q[..., :r] @ p["dt_proj"].t()
    y, ss = R.scan(u, delta, -torch.exp(p["A_log"]), q[..., r:r + n].unsqueeze(2), q[..., r + n:].unsqueeze(2), p["D"],
                   xz[..., d:], p["dt_bias"], None if state is None else state[1], lengths)
    return x + y @ p["out_proj"].t(), (cs, ss), p


@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_through_a_block(ragged):
    """float32, tolerance: the operators' own (2e-4 of the largest value), through four products
    of at most 128 terms each (128 * 2^-24 of their terms' sizes, a few times the result's)."""
    torch.manual_seed(3)
    block = SelectiveBlock(48, dstate=16, rank=4, dtype=torch.float32, device=DEV)
    x = torch.randn(3, 70, 48)
    dy = torch.randn(3, 70, 48)
    lengths = torch.tensor([70, 0, 33], dtype=torch.int32) if ragged else None
    if ragged:       # the residual passes tokens past a row's end through; leave them out of the loss
        for i, m in enumerate(lengths.tolist()):
            dy[i, m:] = 0
    xg = x.to(DEV).requires_grad_(True)
    y, state = block(xg, lengths=None if lengths is None else lengths.to(DEV))
    (y * dy.to(DEV)).sum().backward()
    torch.cuda.synchronize()
    xr = R.up(x).requires_grad_(True)
    yr, sr, p = reference(block, xr, None, lengths)
    grads = R.grads((yr,), (R.up(dy),), [xr] + list(p.values()))
    R.check(y, yr, torch.float32, 4e-4, "y")
    R.check(state[0], sr[0], torch.float32, 4e-4, "convolution state")
    R.check(state[1], sr[1], torch.float32, 4e-4, "scan state")
    R.check(xg.grad, grads[0], torch.float32, 4e-4, "x")
    for (name, q), g in zip(block.named_parameters(), grads[1:]):
        R.check(q.grad, g, torch.float32, 4e-4, name)


def test_prompt_then_tokens():
    """bfloat16: the same roundings in both, so the prompt's outputs and the steps' differ by the
    matrix products' order of addition alone; 2e-2 of the largest value, as for the scans."""
    torch.manual_seed(4)
    block = SelectiveBlock(96, device=DEV)
    x = torch.randn(5, 60, 96, device=DEV).bfloat16()
    with torch.no_grad():
        whole, end = block(x)
        y, state = block(x[:, :41].contiguous())
        ys = [block.step(x[:, t], state) for t in range(41, 60)]
    torch.cuda.synchronize()
    got = torch.cat([y, torch.stack(ys, 1)], 1)
    assert float((got.float() - whole.float()).abs().max()) <= 2e-2 * float(whole.float().abs().max())
    for a, b in zip(state, end):
        assert float((a.float() - b.float()).abs().max()) <= 2e-2 * float(b.float().abs().max())


def test_state_carries_gradients():
    """A sequence in two parts, the second starting from the first's states: gradients reach the
    first part through the states as in one call."""
    torch.manual_seed(5)
    block = SelectiveBlock(32, rank=2, dtype=torch.float32, device=DEV)
    x = torch.randn(2, 50, 32, device=DEV)
    dy = torch.randn(2, 50, 32, device=DEV)
    grads = []
    for cut in (None, 23):
        xa = x.clone().requires_grad_(True)
        if cut is None:
            y, _ = block(xa)
        else:
            y1, state = block(xa[:, :cut])
            y2, _ = block(xa[:, cut:], state)
            y = torch.cat([y1, y2], 1)
        block.zero_grad()
        (y * dy).sum().backward()
        grads.append([xa.grad] + [p.grad.clone() for p in block.parameters()])
    torch.cuda.synchronize()
    for a, b in zip(*grads):
        R.check(a, b, torch.float32, 4e-4, "gradient")


def test_decode_step_in_a_graph():
    """The single-token path captured and replayed, with eager work between the replays, gives
    the eager results bit for bit."""
    torch.manual_seed(6)
    block = SelectiveBlock(64, device=DEV)
    x = torch.randn(3, 64, device=DEV).bfloat16()
    with torch.no_grad():
        _, first = block(torch.randn(3, 9, 64, device=DEV).bfloat16())
    state = tuple(t.clone() for t in first)
    ref = [block.step(x, state).clone() for _ in range(3)]
    ref_state = [t.clone() for t in state]
    static = tuple(t.clone() for t in first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.step(x, static)
    for t, f in zip(static, first):
        t.copy_(f)
    for k in range(3):
        torch.randn(100, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[k]), k
    for a, b in zip(static, ref_state):
        assert torch.equal(a, b)


def test_stale_state_and_second_derivatives_are_refused():
    """A backward whose incoming state a step has overwritten since, and a derivative of a
    gradient, which the kernels do not have, raise instead of giving wrong values."""
    torch.manual_seed(7)
    block = SelectiveBlock(32, rank=2, dtype=torch.float32, device=DEV)
    x = torch.randn(2, 9, 32, device=DEV)
    with torch.no_grad():
        _, state = block(x)
    y, _ = block(x, state)
    block.step(x[:, 0], state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    xg = x.clone().requires_grad_(True)
    (dx,) = torch.autograd.grad(block(xg)[0].square().sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()
