"""A selective block from the library's operators: layer norm, in-projection, short causal
convolution with SiLU, selective scan gated by the projection's other half, out-projection,
and the residual.

    block = SelectiveBlock(768, device="cuda")
    y, state = block(x)                  # a prompt [b, L, 768], with gradients
    y_t = block.step(x_t, state)         # the next token [b, 768], the state moved on in place

The projections are plain matrix products (torch); everything between them runs in the
library's kernels, forwards and backwards.  `python -m chunked_linear_recurrence_amd.block`
trains a small block, runs a prompt and continues it token by token.
"""
import math

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import ssd


def _rows(g, like):
    """A gradient as the operators take it: channels contiguous, zeros where there is none."""
    if g is None:
        return torch.zeros_like(like)
    return g if g.stride(-1) == 1 else g.contiguous()


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ssd.norm_fwd(x, weight, bias, eps, want_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = ssd.norm_bwd(_rows(dy, x), x, weight, mean, rstd)
        return g.dx, None if weight is None else g.dweight, g.dbias if ctx.has_bias else None, None


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, init_state, lengths):
        ctx.set_materialize_grads(False)
        y, final = ssd.conv_fwd(x, weight, bias, init_state, lengths=lengths)
        ctx.save_for_backward(x, weight, bias, init_state, lengths)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, init_state, lengths = ctx.saved_tensors
        g = ssd.conv_bwd(_rows(dy, x), x, weight, bias, init_state,
                         dfinal=None if dfinal is None else dfinal.contiguous(), lengths=lengths)
        return g.dx, g.dweight, g.dbias, g.dinit, None


class _Selective(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, init_state, lengths):
        ctx.set_materialize_grads(False)
        y, final, kept = ssd.selective_fwd(u, delta, A, B, C, D, z, delta_bias, init_state, lengths=lengths, keep=True)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, kept, lengths)
        ctx.has_init = init_state is not None
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        u, delta, A, B, C, D, z, delta_bias, kept, lengths = ctx.saved_tensors
        g = ssd.selective_bwd(_rows(dy, u), u, delta, A, B, C, D, z, delta_bias, kept,
                              dfinal=None if dfinal is None else dfinal.contiguous(), lengths=lengths)
        return (g.du, g.ddelta, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddelta_bias, g.dinit if ctx.has_init else None, None)


def norm(x, weight=None, bias=None, eps=1e-5):
    """ssd.norm_fwd with gradients: x [rows, channels]."""
    return _Norm.apply(x, weight, bias, eps)


def conv(x, weight, bias=None, init_state=None, lengths=None):
    """ssd.conv_fwd (with SiLU) with gradients; (y, final_state)."""
    return _Conv.apply(x, weight, bias, init_state, lengths)


def selective(u, delta, A, B, C, D=None, z=None, delta_bias=None, init_state=None, lengths=None):
    """ssd.selective_fwd with gradients; (y, final_state).  The states that the backward needs are
    kept by every call (dstate / 2 bytes a token and channel), with gradients switched off too;
    ssd.selective_fwd by itself keeps none."""
    return _Selective.apply(u, delta, A, B, C, D, z, delta_bias, init_state, lengths)


class SelectiveBlock(torch.nn.Module):
    """Activations and projections are `dtype`; the norm's, convolution's and scan's parameters
    are float32.  rank: channels of the low-rank step size (even, so that B and C behind it in
    one projection's output lie on 4 bytes)."""

    def __init__(self, width, *, expand=2, dstate=16, taps=4, rank=None, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        d, n = expand * width, dstate
        rank = rank if rank is not None else 2 * math.ceil(width / 32)
        if rank % 2:
            raise ValueError("rank must be even (got %d)" % rank)
        self.width, self.channels, self.dstate, self.taps, self.rank = width, d, n, taps, rank

        def matrix(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, device=device) / math.sqrt(cols)).to(dtype))

        def f32(t):
            return torch.nn.Parameter(t.to(device=device, dtype=torch.float32))
        self.norm_weight, self.norm_bias = f32(torch.ones(width)), f32(torch.zeros(width))
        self.in_proj = matrix(2 * d, width)
        self.conv_weight, self.conv_bias = f32(torch.randn(d, taps) / math.sqrt(taps)), f32(torch.zeros(d))
        self.x_proj = matrix(rank + 2 * n, d)
        self.dt_proj = matrix(d, rank)
        # step sizes spread over [1e-3, 0.1] at the start, decay rates 1..N
        dt0 = torch.exp(torch.rand(d) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = f32(dt0 + torch.log(-torch.expm1(-dt0)))
        self.A_log = f32(torch.log(torch.arange(1, n + 1).float()).repeat(d, 1))
        self.D = f32(torch.ones(d))
        self.out_proj = matrix(width, d)

    def forward(self, x, state=None, lengths=None):
        """x [b, L, width]; state as returned (None: zeros); lengths [b] int32: each row's own
        tokens.  What x holds past them reaches no result and no gradient but the residual's own.
        Returns (y [b, L, width], state)."""
        b, L, _ = x.shape
        d, n, r = self.channels, self.dstate, self.rank
        conv_state, scan_state = state if state is not None else (None, None)
        own = x
        if lengths is not None:      # the norm and the projections take every row; 0 x NaN would reach their weights
            own = x.masked_fill((torch.arange(L, device=x.device) >= lengths[:, None])[..., None], 0)
        h = norm(own.reshape(b * L, self.width), self.norm_weight, self.norm_bias)
        xz = F.linear(h, self.in_proj).view(b, L, 2 * d)
        u, conv_state = conv(xz[..., :d], self.conv_weight, self.conv_bias, conv_state, lengths)
        p = F.linear(u.view(b * L, d), self.x_proj)
        delta = F.linear(p[:, :r], self.dt_proj).view(b, L, d)
        B = p[:, r:r + n].view(b, L, 1, n)
        C = p[:, r + n:].view(b, L, 1, n)
        y, scan_state = selective(u, delta, -torch.exp(self.A_log), B, C, self.D, xz[..., d:], self.dt_bias, scan_state,
                                  lengths)
        return x + F.linear(y.view(b * L, d), self.out_proj).view(b, L, self.width), (conv_state, scan_state)

    @torch.no_grad()
    def step(self, x, state):
        """One token x [b, width]; state is moved on in place.  Returns y [b, width]."""
        d, n, r = self.channels, self.dstate, self.rank
        h = ssd.norm_fwd(x, self.norm_weight, self.norm_bias)
        xz = F.linear(h, self.in_proj)
        u = ssd.conv_step(xz[:, :d], self.conv_weight, self.conv_bias, state[0])
        p = F.linear(u, self.x_proj)
        delta = F.linear(p[:, :r], self.dt_proj)
        y = ssd.selective_step(u, delta, -torch.exp(self.A_log), p[:, None, r:r + n], p[:, None, r + n:], self.D, xz[:, d:],
                               self.dt_bias, state[1])
        return x + F.linear(y, self.out_proj)


def main():
    torch.manual_seed(0)
    b, L, width, T = 4, 512, 256, 32
    block = SelectiveBlock(width)
    opt = torch.optim.Adam(block.parameters(), lr=2e-3)
    x = torch.randn(b, L, width, device="cuda").bfloat16()
    target = torch.roll(x, 3, 1)                       # each token answers with the one three before it
    for k in range(20):
        y, _ = block(x)
        loss = (y.float() - target.float())[:, 3:].square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        if k % 5 == 0 or k == 19:
            print("training step %2d: loss %.4f" % (k, loss.item()), flush=True)
    with torch.no_grad():
        whole, _ = block(x)
        y, state = block(x[:, :L - T].contiguous())
        steps = [block.step(x[:, t], state) for t in range(L - T, L)]
        err = (torch.stack(steps, 1).float() - whole[:, L - T:].float()).abs().max().item()
    print("prompt of %d tokens, then %d single tokens: largest difference from one prompt %.3g (largest value %.3g)" % (
        L - T, T, err, whole.float().abs().max().item()), flush=True)


if __name__ == "__main__":
    main()
