"""A selective block from the library's operators: layer norm, in-projection, short causal
convolution with SiLU, selective scan gated by the projection's other half, out-projection,
and the residual.

    block = SelectiveBlock(768, device="cuda")
    y, state = block(x)                  # a prompt [b, L, 768], with gradients
    y_t = block.step(x_t, state)         # the next token [b, 768], the state moved on in place

The projections are plain matrix products (torch); everything between them runs in the
library's kernels, forwards and backwards.

    layer = SelectiveLayer(768, device="cuda")

is such a block and a gated feed-forward behind it, called in the same way: the sum with the
residual and the norm between the two halves are one kernel, the gated product one, and the
product back with its residual one.  `python -m chunked_linear_recurrence_amd.block` trains a
small block and a small layer, runs a prompt of each and continues it token by token.
"""
import math

import torch
import torch.nn.functional as F
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import ssd


def _rows(g, like):
    """A gradient as the operators take it: channels contiguous, zeros where there is none."""
    if g is None:
        return torch.zeros_like(like)
    return g if g.stride(-1) == 1 else g.contiguous()


def _last_contiguous(g):
    return g if g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous()


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


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act):
        y, pre = ssd.linear_fwd(x, weight, bias, residual, act=act, keep=True)
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.act = act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, pre = ctx.saved_tensors
        g = ssd.linear_bwd(_last_contiguous(dy), x, weight, bias, pre, act=ctx.act, need=ctx.needs_input_grad[:3])
        return g.dx, g.dweight, g.dbias, dy if ctx.needs_input_grad[3] else None, None


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, act):
        h, pre = ssd.gated_fwd(x, weight, bias, act=act, keep=True)
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.act = act
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, weight, bias, pre = ctx.saved_tensors
        g = ssd.gated_bwd(_last_contiguous(dh), x, weight, bias, pre, act=ctx.act, need=ctx.needs_input_grad[:3])
        return g.dx, g.dweight, g.dbias, None


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, branch, residual, gate, post_weight, scale, pre_weight, eps):
        ctx.set_materialize_grads(False)
        y, total, stats = ssd.residual_norm_fwd(branch, residual, gate, post_weight, scale, pre_weight, eps, want_stats=True)
        ctx.save_for_backward(branch, residual, gate, post_weight, scale, pre_weight, stats)
        return y, total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dtotal):
        branch, residual, gate, post_weight, scale, pre_weight, stats = ctx.saved_tensors
        dy = None if pre_weight is None else _rows(dy, branch)
        if dtotal is not None or dy is None:
            dtotal = _rows(dtotal, branch)
        g = ssd.residual_norm_bwd(dy, dtotal, branch, residual, gate, post_weight, scale, pre_weight, stats)
        return g.dbranch, g.dresidual, g.dgate, g.dpost_weight, g.dscale, g.dpre_weight, None


def _differentiated(*tensors):
    """Whether a backward can follow a call on these tensors (others are left to the call's own
    checks), or a tangent comes with one, which the functions with gradients refuse."""
    given = [t for t in tensors if isinstance(t, torch.Tensor)]
    return (torch.is_grad_enabled() and any(t.requires_grad for t in given)) or any(
        forward_ad.unpack_dual(t).tangent is not None for t in given)


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


def linear(x, weight, bias=None, residual=None, act=None):
    """ssd.linear_fwd with gradients: x [rows, inner], weight [outer, inner].  What a backward needs is
    kept where one can follow: gradients are enabled and an input requires them."""
    if not _differentiated(x, weight, bias, residual):
        return ssd.linear_fwd(x, weight, bias, residual, act=act)
    return _Linear.apply(x, weight, bias, residual, act)


def gated(x, weight, bias=None, act="silu"):
    """ssd.gated_fwd with gradients: x [rows, inner], weight [2 hidden, inner].  What a backward needs
    (2 hidden values a row) is kept as by linear."""
    if not _differentiated(x, weight, bias):
        return ssd.gated_fwd(x, weight, bias, act=act)
    return _Gated.apply(x, weight, bias, act)


def residual_norm(branch, residual=None, gate=None, post_weight=None, scale=None, pre_weight=None, eps=1e-5):
    """ssd.residual_norm_fwd with gradients; (y, total), y None without pre_weight."""
    if not _differentiated(branch, residual, gate, post_weight, scale, pre_weight):
        return ssd.residual_norm_fwd(branch, residual, gate, post_weight, scale, pre_weight, eps)
    return _ResidualNorm.apply(branch, residual, gate, post_weight, scale, pre_weight, eps)


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

    def branch(self, x, state=None, lengths=None):
        """What forward adds to x, [b * L, width], and the state."""
        b, L, _ = x.shape
        d, n, r = self.channels, self.dstate, self.rank
        conv_state, scan_state = state if state is not None else (None, None)
        own = x
        if lengths is not None:      # the norm and the projections take every row; 0 x NaN would reach their weights
            own = x.masked_fill(_behind(x, lengths), 0)
        h = norm(own.reshape(b * L, self.width), self.norm_weight, self.norm_bias)
        xz = F.linear(h, self.in_proj).view(b, L, 2 * d)
        u, conv_state = conv(xz[..., :d], self.conv_weight, self.conv_bias, conv_state, lengths)
        p = F.linear(u.view(b * L, d), self.x_proj)
        delta = F.linear(p[:, :r], self.dt_proj).view(b, L, d)
        B = p[:, r:r + n].view(b, L, 1, n)
        C = p[:, r + n:].view(b, L, 1, n)
        y, scan_state = selective(u, delta, -torch.exp(self.A_log), B, C, self.D, xz[..., d:], self.dt_bias, scan_state,
                                  lengths)
        return F.linear(y.view(b * L, d), self.out_proj), (conv_state, scan_state)

    def forward(self, x, state=None, lengths=None):
        """x [b, L, width]; state as returned (None: zeros); lengths [b] int32: each row's own
        tokens.  What x holds past them reaches no result and no gradient but the residual's own.
        Returns (y [b, L, width], state)."""
        y, state = self.branch(x, state, lengths)
        return x + y.view(x.shape), state

    @torch.no_grad()
    def step_branch(self, x, state):
        """What step adds to x."""
        d, n, r = self.channels, self.dstate, self.rank
        h = ssd.norm_fwd(x, self.norm_weight, self.norm_bias)
        xz = F.linear(h, self.in_proj)
        u = ssd.conv_step(xz[:, :d], self.conv_weight, self.conv_bias, state[0])
        p = F.linear(u, self.x_proj)
        delta = F.linear(p[:, :r], self.dt_proj)
        y = ssd.selective_step(u, delta, -torch.exp(self.A_log), p[:, None, r:r + n], p[:, None, r + n:], self.D, xz[:, d:],
                               self.dt_bias, state[1])
        return F.linear(y, self.out_proj)

    @torch.no_grad()
    def step(self, x, state):
        """One token x [b, width]; state is moved on in place.  Returns y [b, width]."""
        return x + self.step_branch(x, state)


def _behind(x, lengths):
    """[b, L, 1]: the tokens behind each row's own."""
    return (torch.arange(x.shape[1], device=x.device) >= lengths[:, None])[..., None]


class SelectiveLayer(torch.nn.Module):
    """A SelectiveBlock and a gated feed-forward of `hidden` channels (8/3 of the width, a whole
    number of 64, by default) behind it:
        total = x + scale * branch(x);  y = total + out(act(g) * u),  [g | u] = rms(total) w_in^T
    scale [width] and the norm's weight are float32, the projections `dtype`.  Arguments beside
    these are the block's."""

    def __init__(self, width, hidden=None, *, act="silu", dtype=torch.bfloat16, device="cuda", **block):
        super().__init__()
        self.block = SelectiveBlock(width, dtype=dtype, device=device, **block)
        self.width, self.hidden, self.act = width, hidden or 64 * math.ceil(width / 24), act
        self.scale = torch.nn.Parameter(torch.ones(width, device=device))
        self.norm_weight = torch.nn.Parameter(torch.ones(width, device=device))

        def matrix(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, device=device) / math.sqrt(cols)).to(dtype))
        self.in_proj, self.out_proj = matrix(2 * self.hidden, width), matrix(width, self.hidden)

    def forward(self, x, state=None, lengths=None):
        """As SelectiveBlock's, but the outputs behind a row's own tokens are 0 and what x holds
        there reaches no gradient at all."""
        b, L, _ = x.shape
        if lengths is not None:
            x = x.masked_fill(_behind(x, lengths), 0)
        branch, state = self.block.branch(x, state, lengths)
        n, total = residual_norm(branch, x.reshape(b * L, self.width), scale=self.scale, pre_weight=self.norm_weight)
        y = linear(gated(n, self.in_proj, act=self.act), self.out_proj, residual=total)
        return y.view(b, L, self.width), state

    @torch.no_grad()
    def step(self, x, state):
        """One token x [b, width]; state is moved on in place.  Returns y [b, width]."""
        n, total = ssd.residual_norm_fwd(self.block.step_branch(x, state), x, scale=self.scale, pre_weight=self.norm_weight)
        return ssd.linear_fwd(ssd.gated_fwd(n, self.in_proj, act=self.act), self.out_proj, None, total)


def _train(name, model, max_norm=None):
    """Trains on a small task, then runs a prompt and continues it token by token."""
    b, L, width, T = 4, 512, model.width, 32
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    x = torch.randn(b, L, width, device="cuda").bfloat16()
    target = torch.roll(x, 3, 1)                       # each token answers with the one three before it
    for k in range(20):
        y, _ = model(x)
        loss = (y.float() - target.float())[:, 3:].square().mean()
        opt.zero_grad()
        loss.backward()
        norm = None if max_norm is None else ssd.clip_grads([p.grad for p in model.parameters()], max_norm)
        opt.step()
        if k % 5 == 0 or k == 19:
            print("%s, training step %2d: loss %.4f%s" % (
                name, k, loss.item(), "" if norm is None else ", gradients' norm %.4f" % norm.item()), flush=True)
    with torch.no_grad():
        whole, _ = model(x)
        y, state = model(x[:, :L - T].contiguous())
        steps = [model.step(x[:, t], state) for t in range(L - T, L)]
        err = (torch.stack(steps, 1).float() - whole[:, L - T:].float()).abs().max().item()
    print("%s, prompt of %d tokens, then %d single tokens: largest difference from one prompt %.3g (largest value %.3g)" % (
        name, L - T, T, err, whole.float().abs().max().item()), flush=True)


def main():
    torch.manual_seed(0)
    _train("block", SelectiveBlock(256))
    _train("layer", SelectiveLayer(256), max_norm=0.1)


if __name__ == "__main__":
    main()
