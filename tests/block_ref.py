"""Plain float64 references of the operators around a scan (short convolution, selective
scan, layer norm), written token by token from their definitions, with gradients by
differentiation; and the comparison their tests use."""
import torch

F64 = torch.float64


def check(got, ref, dtype, tol, what="", scale=0.0):
    """|got - ref| <= tol max(max|ref|, scale) (+ 2^-8 |ref| where the result is stored in bfloat16);
    scale is the size of the terms where they cancel in every element."""
    g, r = got.detach().cpu().to(F64), ref.detach().cpu().to(F64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert torch.isfinite(g).all(), what + " has values that are not finite"
    if r.numel() == 0:
        return
    bound = tol * max(float(r.abs().max()), scale) + (2.0 ** -8 * r.abs() if dtype == torch.bfloat16 else 0.0)
    over = ((g - r).abs() - bound).max()
    assert over <= 0, "%s: off by %.3g beyond its bound (max |ref| %.3g)" % (what, over, r.abs().max())


def up(t):
    return None if t is None else t.detach().cpu().to(F64)


def lens_of(lengths, b, L):
    return [L] * b if lengths is None else [max(0, min(int(v), L)) for v in lengths]


def conv(x, w, bias=None, init=None, lengths=None, silu=True):
    """(y, final) of float64 tensors on the CPU, row by row."""
    b, L, C = x.shape
    W = w.shape[1]
    ys, fs = [], []
    for i, m in enumerate(lens_of(lengths, b, L)):
        head = init[i] if init is not None else torch.zeros(W - 1, C, dtype=F64)
        row = torch.cat([head, x[i, :m]], 0)
        pre = torch.zeros(m, C, dtype=F64) if bias is None else bias.expand(m, C)
        for j in range(W):
            pre = pre + row[j:j + m] * w[:, j]
        y = pre * torch.sigmoid(pre) if silu else pre
        ys.append(torch.cat([y, torch.zeros(L - m, C, dtype=F64)], 0))
        fs.append(row[m:m + W - 1])
    return torch.stack(ys), torch.stack(fs)


def scan(u, delta, A, B, C, D=None, z=None, bias=None, init=None, lengths=None, softplus=True):
    """(y, final) of float64 tensors on the CPU, token by token."""
    b, L, d = u.shape
    G, N = B.shape[2:]
    grp = torch.arange(d) // (d // G)
    outs, finals = [], []
    for i, m in enumerate(lens_of(lengths, b, L)):
        h = init[i] if init is not None else torch.zeros(d, N, dtype=F64)
        ys = []
        for t in range(m):
            dt = delta[i, t] + (bias if bias is not None else 0.0)
            if softplus:
                dt = torch.nn.functional.softplus(dt, threshold=1e9) if dt.max() < 700 else torch.log1p(dt.exp())
            h = torch.exp(dt[:, None] * A) * h + (dt * u[i, t])[:, None] * B[i, t][grp]
            y = (h * C[i, t][grp]).sum(1)
            if D is not None:
                y = y + D * u[i, t]
            if z is not None:
                y = y * z[i, t] * torch.sigmoid(z[i, t])
            ys.append(y)
        y = torch.stack(ys) if ys else torch.zeros(0, d, dtype=F64)
        outs.append(torch.cat([y, torch.zeros(L - m, d, dtype=F64)], 0))
        finals.append(h)
    return torch.stack(outs), torch.stack(finals)


def norm(x, w=None, b=None, eps=1e-5):
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps)
    y = xc * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean[:, 0], rstd[:, 0]


def grads(outs, cotangents, leaves):
    """Gradients of sum(out * cotangent) by each leaf (zeros where it does not enter)."""
    loss = sum((o * c).sum() for o, c in zip(outs, cotangents) if c is not None)
    if not loss.requires_grad:
        return [torch.zeros_like(t) for t in leaves]
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(t) if v is None else v for v, t in zip(g, leaves)]
