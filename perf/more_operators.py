"""The operators of a layer's feed-forward half and of its training step, as they are measured:
the matrix product with bias, activation and residual in its epilogue, the gated feed-forward
product, the norms after and before a block fused with its gate and residual scale, and the
clipping of gradients by their global norm.

`run` computes them in elementary torch operations (32 bits, rounded once at the end) where
`own` is false, and calls the package's entry points where it is true; `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decoded token through the out-projection of a 1024-wide block (expand 2), with
        # the residual: latency of the call.
        dict(name="linear_prompt_r1_k2048_n1024", op="linear_prompt", rows=1, inner=2048, outer=1024, dtype="bf16",
             act="none", bias=False, residual=True),
        # The out-projection over 8 prompts of 4096 tokens, with the residual.
        dict(name="linear_prompt_r32768_k4096_n2048", op="linear_prompt", rows=32768, inner=4096, outer=2048,
             dtype="bf16", act="none", bias=False, residual=True),
        # A training step of a projection with bias and activation, float32, odd everywhere.
        dict(name="linear_train_r1999_k777_n1025_f32", op="linear_train", rows=1999, inner=777, outer=1025, dtype="f32",
             act="silu", bias=True, residual=True),
        # One decoded token through the gated product: latency, and the weights' traffic.
        dict(name="gated_prompt_r1_k768_f2048", op="gated_prompt", rows=1, inner=768, outer=2048, dtype="bf16",
             act="silu", bias=False),
        # One token for each of 48 streams.
        dict(name="gated_prompt_r48_k2048_f5632", op="gated_prompt", rows=48, inner=2048, outer=5632, dtype="bf16",
             act="silu", bias=False),
        # An ordinary prompt (one 2048-token segment).
        dict(name="gated_prompt_r2048_k1536_f4096", op="gated_prompt", rows=2048, inner=1536, outer=4096, dtype="bf16",
             act="silu", bias=False),
        # A training step over two rows of 4096 tokens.
        dict(name="gated_train_r8192_k2048_f5632", op="gated_train", rows=8192, inner=2048, outer=5632, dtype="bf16",
             act="silu", bias=True),
        # One decoded token: the sum with the residual and the next block's norm.
        dict(name="residual_norm_prompt_r1_d768", op="residual_norm_prompt", rows=1, chan=768, dtype="bf16",
             gate=False, post=False, scale=False),
        # A training step over 8 x 4096 tokens: gate, norm after the block, scale, sum, next norm.
        dict(name="residual_norm_train_r32768_d2048", op="residual_norm_train", rows=32768, chan=2048, dtype="bf16",
             gate=True, post=True, scale=True),
        # A float32 training step of odd sizes.
        dict(name="residual_norm_train_r4099_d1025_f32", op="residual_norm_train", rows=4099, chan=1025, dtype="f32",
             gate=False, post=True, scale=True),
        # The gradients of one small block.
        dict(name="clip_block_w256", op="clip", kind="block", layers=1, width=256, dtype="bf16", over=True),
        # The gradients of a stack of 5 blocks.
        dict(name="clip_stack5_w2048", op="clip", kind="block", layers=5, width=2048, dtype="bf16", over=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    n = _spread(rng, lo, hi)
    return n if rng.random() < 0.5 else max(64, n // 64 * 64)      # half at a multiple of 64, as most widths are


def draw(rng):
    op = rng.choice(["linear_prompt", "linear_train", "gated_prompt", "gated_train", "residual_norm_prompt",
                     "residual_norm_train", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        if rng.random() < 0.5:
            return dict(op=op, kind="block", layers=_spread(rng, 1, 5), width=64 * _spread(rng, 1, 24), dtype=dtype,
                        over=rng.random() < 0.7)
        return dict(op=op, kind="any", count=_spread(rng, 1, 60), largest=_spread(rng, 16, 1 << 20),
                    sizes=rng.randrange(1 << 30), dtype=dtype, over=rng.random() < 0.7)
    if op.startswith("residual_norm"):
        chan = _spread(rng, 64, 8192)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(32768, (1 << 25) // chan))), chan=chan, dtype=dtype,
                    gate=rng.random() < 0.5, post=rng.random() < 0.5, scale=rng.random() < 0.5)
    inner, outer = _size(rng, 64, 8192), _size(rng, 64, 8192)
    room = (1 << 37 if dtype == "bf16" else 1 << 34) // (3 if op.endswith("train") else 1)
    room //= inner * outer * (2 if op.startswith("gated") else 1)
    c = dict(op=op, rows=_spread(rng, 1, max(1, min(32768, room))), inner=inner, outer=outer, dtype=dtype,
             act=rng.choice(["silu", "gelu"]) if op.startswith("gated") else rng.choice(["none", "silu", "gelu"]),
             bias=rng.random() < 0.5)
    if op.startswith("linear"):
        c["residual"] = rng.random() < 0.5
    return c


def _clip_shapes(case):
    """The shapes and types of the tensors of a clip case."""
    if case["kind"] == "block":        # a selective block's: projections in its type, the rest in float32
        w, d, n, r = case["width"], 2 * case["width"], 16, 2 * math.ceil(case["width"] / 32)
        one = [((w,), "f32"), ((w,), "f32"), ((2 * d, w), case["dtype"]), ((d, 4), "f32"), ((d,), "f32"),
               ((r + 2 * n, d), case["dtype"]), ((d, r), case["dtype"]), ((d,), "f32"), ((d, n), "f32"), ((d,), "f32"),
               ((w, d), case["dtype"])]
        return one * case["layers"]
    rng = random.Random(case["sizes"])
    return [((_spread(rng, 1, case["largest"]),), rng.choice([case["dtype"], "f32"])) for _ in range(case["count"])]


def work(case):
    op = case["op"]
    if op == "clip":
        # read for the norm; where it clips, the norm has to be known before the first value is
        # written, so each is read again and written (where it does not, copied)
        n = [(math.prod(s), 2 if t == "bf16" else 4) for s, t in _clip_shapes(case)]
        return {"bytes": sum(3 * k * e for k, e in n), "flops": sum(3 * k for k, _ in n)}
    e = 2 if case["dtype"] == "bf16" else 4
    m = case["rows"]
    if op.startswith("residual_norm"):
        n, ch = m * case["chan"], case["chan"]
        reads = 2 + case["gate"]
        par = 4 * ch * (1 + case["post"] + case["scale"])
        if op == "residual_norm_prompt":
            return {"bytes": (reads + 2) * n * e + par, "flops": n * (5 + 6 * case["gate"] + 4 * case["post"])}
        # forward as above; then both gradients in, those of branch, residual and gate out
        return {"bytes": (reads + 2 + 2 + reads) * n * e + 2 * par + 8 * m,
                "flops": n * (20 + 16 * case["gate"] + 14 * case["post"])}
    k = case["inner"]
    f = case["outer"] * (2 if op.startswith("gated") else 1)
    size = m * k + f * k + m * case["outer"] + (f if case["bias"] else 0) + (m * f if case.get("residual") else 0)
    if op.endswith("prompt"):
        return {"bytes": size * e, "flops": 2 * m * k * f}
    # the output's gradient in; those of x, weight and bias out
    size += m * case["outer"] + m * k + f * k + (f if case["bias"] else 0)
    return {"bytes": size * e, "flops": 6 * m * k * f}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]

    def randn(*shape, std=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype or _DT[case["dtype"]])

    s = {"case": case}
    if op == "clip":
        shapes = _clip_shapes(case)
        s["grads"] = [randn(*shape, std=10.0 ** -(1 + k % 4), dtype=_DT[t]) for k, (shape, t) in enumerate(shapes)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        # spread of the sum of squares by construction: clipped by about two, or not at all
        size = math.sqrt(sum(math.prod(shape) * 100.0 ** -(1 + k % 4) for k, (shape, _) in enumerate(shapes)))
        s["max_norm"] = size * (0.5 if case["over"] else 4.0)
        return s
    m = case["rows"]
    if op.startswith("residual_norm"):
        ch = case["chan"]
        s["branch"], s["residual"] = randn(m, ch), randn(m, ch, std=2.0)
        s["gate"] = randn(m, ch) if case["gate"] else None
        s["post"] = 1.0 + 0.2 * randn(ch, dtype=torch.float32) if case["post"] else None
        s["scale"] = 0.5 + 0.2 * randn(ch, dtype=torch.float32) if case["scale"] else None
        s["pre"] = 1.0 + 0.2 * randn(ch, dtype=torch.float32)
        if op.endswith("train"):
            s["dy"], s["dtotal"] = randn(m, ch), randn(m, ch)
        return s
    k, n = case["inner"], case["outer"]
    f = 2 * n if op.startswith("gated") else n
    s["x"] = randn(m, k)
    s["weight"] = randn(f, k, std=1.0 / math.sqrt(k))
    s["bias"] = randn(f, std=0.2) if case["bias"] else None
    s["residual"] = randn(m, n) if case.get("residual") else None
    if op.endswith("train"):
        s["dy"] = randn(m, n)
    return s


# ---------------------------------------------------------------------- the plain forms
def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    return v


def _dact(v, act):
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return sig * (1.0 + v * (1.0 - sig))
    if act == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(v)


def _plain_linear(s, train):
    x, w, act = s["x"].float(), s["weight"].float(), s["case"]["act"]
    dt = s["x"].dtype
    pre = x @ w.t()
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    y = _act(pre, act)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(dt)
    if not train:
        return y
    dpre = s["dy"].float() * _dact(pre, act)
    out = (y, (dpre @ w).to(dt), (dpre.t() @ x).to(dt))
    return out + ((dpre.sum(0).to(dt),) if s["bias"] is not None else ())


def _plain_gated(s, train):
    x, w, act = s["x"].float(), s["weight"].float(), s["case"]["act"]
    dt, f = s["x"].dtype, s["weight"].shape[0] // 2
    pre = x @ w.t()
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    g, u = pre[:, :f], pre[:, f:]
    a = _act(g, act)
    h = (a * u).to(dt)
    if not train:
        return h
    dh = s["dy"].float()
    dpre = torch.cat([dh * u * _dact(g, act), dh * a], 1)
    out = (h, (dpre @ w).to(dt), (dpre.t() @ x).to(dt))
    return out + ((dpre.sum(0).to(dt),) if s["bias"] is not None else ())


def _rms(v):
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)
    return v * rstd, rstd


def _plain_residual_norm(s, train):
    branch, residual = s["branch"].float(), s["residual"].float()
    dt = s["branch"].dtype
    t = branch
    if s["gate"] is not None:
        z = s["gate"].float()
        t = branch * _act(z, "silu")
    p = t
    if s["post"] is not None:
        that, rt = _rms(t)
        p = that * s["post"]
    total = residual + (p * s["scale"] if s["scale"] is not None else p)
    shat, rs = _rms(total)
    y = shat * s["pre"]
    out = (y.to(dt), total.to(dt))
    if not train:
        return out
    dy = s["dy"].float()
    g = dy * s["pre"]
    ds = s["dtotal"].float() + rs * (g - shat * (g * shat).mean(1, keepdim=True))
    dpre = (dy * shat).sum(0)
    dp = ds * s["scale"] if s["scale"] is not None else ds
    dscale = (ds * p).sum(0)
    dpost = None
    d = dp
    if s["post"] is not None:
        dpost = (dp * that).sum(0)
        g = dp * s["post"]
        d = rt * (g - that * (g * that).mean(1, keepdim=True))
    out += (ds.to(dt), dpre)
    if s["scale"] is not None:
        out += (dscale,)
    if s["post"] is not None:
        out += (dpost,)
    if s["gate"] is None:
        return out + (d.to(dt),)
    return out + ((d * _act(z, "silu")).to(dt), (d * branch * _dact(z, "silu")).to(dt))


def _plain_clip(s):
    total = sum((g.float() * g.float()).sum(dtype=torch.float64) for g in s["grads"])
    norm = torch.sqrt(total)
    factor = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    return (norm.float(),) + tuple((g.float() * factor).to(g.dtype) for g in s["grads"])


# ------------------------------------------------------------------------------ a pass
def run(state):
    s = state
    op = s["case"]["op"]
    train = op.endswith("train")
    if not own:
        if op == "clip":
            return _plain_clip(s)
        if op.startswith("residual_norm"):
            return _plain_residual_norm(s, train)
        return _plain_linear(s, train) if op.startswith("linear") else _plain_gated(s, train)
    from chunked_linear_recurrence_amd import ssd
    if op == "clip":
        norm = ssd.clip_grads(s["grads"], s["max_norm"], out=s["out"])
        return (norm,) + tuple(s["out"])
    if op.startswith("residual_norm"):
        args = (s["branch"], s["residual"], s["gate"], s["post"], s["scale"], s["pre"])
        if not train:
            return ssd.residual_norm_fwd(*args, eps=_EPS)
        y, total, stats = ssd.residual_norm_fwd(*args, eps=_EPS, want_stats=True)
        g = ssd.residual_norm_bwd(s["dy"], s["dtotal"], *args, stats)
        out = (y, total, g.dresidual, g.dpre_weight)
        if s["scale"] is not None:
            out += (g.dscale,)
        if s["post"] is not None:
            out += (g.dpost_weight,)
        return out + ((g.dbranch,) if s["gate"] is None else (g.dbranch, g.dgate))
    act = None if s["case"]["act"] == "none" else s["case"]["act"]
    if op == "linear_prompt":
        return ssd.linear_fwd(s["x"], s["weight"], s["bias"], s["residual"], act=act)
    if op == "linear_train":
        y, pre = ssd.linear_fwd(s["x"], s["weight"], s["bias"], s["residual"], act=act, keep=True)
        g = ssd.linear_bwd(s["dy"], s["x"], s["weight"], s["bias"], pre, act=act)
        return (y, g.dx, g.dweight) + (() if s["bias"] is None else (g.dbias,))
    if op == "gated_prompt":
        return ssd.gated_fwd(s["x"], s["weight"], s["bias"], act=act)
    h, pre = ssd.gated_fwd(s["x"], s["weight"], s["bias"], act=act, keep=True)
    g = ssd.gated_bwd(s["dy"], s["x"], s["weight"], s["bias"], pre, act=act)
    return (h, g.dx, g.dweight) + (() if s["bias"] is None else (g.dbias,))


# ------------------------------------------------------------------- the definitions, 64 bits
def _phi(v, act):
    """The activations by their definitions: v times the logistic or the normal distribution."""
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return v


def _exact_product(s, op):
    leaves = [s["x"].double(), s["weight"].double()] + ([] if s["bias"] is None else [s["bias"].double()])
    train, act = op.endswith("train"), s["case"]["act"]
    for t in leaves:
        t.requires_grad_(train)
    with torch.set_grad_enabled(train):
        pre = torch.mm(leaves[0], leaves[1].t())
        if s["bias"] is not None:
            pre = pre + leaves[2]
        if op.startswith("gated"):
            gate, up = pre.chunk(2, 1)
            y = _phi(gate, act) * up
        else:
            y = _phi(pre, act)
            if s["residual"] is not None:
                y = y + s["residual"].double()
        if train:
            grads = torch.autograd.grad(y, leaves, s["dy"].double())
    return (y.detach(),) + tuple(grads) if train else y


def _exact_residual_norm(s, train):
    names = ["branch", "residual"] + [k for k in ("gate", "post", "scale") if s[k] is not None] + ["pre"]
    v = {k: s[k].double().requires_grad_(train) for k in names}

    def rms(t):
        return t / torch.sqrt((t ** 2).mean(1, keepdim=True) + _EPS)
    with torch.set_grad_enabled(train):
        t = v["branch"]
        if "gate" in v:
            t = t * torch.nn.functional.silu(v["gate"])
        if "post" in v:
            t = rms(t) * v["post"]
        if "scale" in v:
            t = t * v["scale"]
        total = v["residual"] + t
        y = rms(total) * v["pre"]
        if train:
            order = ["residual", "pre"] + [k for k in ("scale", "post") if k in v] + ["branch"] + (
                ["gate"] if "gate" in v else [])
            grads = torch.autograd.grad((y, total), [v[k] for k in order], (s["dy"].double(), s["dtotal"].double()))
    return (y.detach(), total.detach()) + (tuple(grads) if train else ())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        factor = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
        return (torch.tensor(norm, dtype=torch.float64, device="cuda"),) + tuple(g.double() * factor for g in s["grads"])
    if op.startswith("residual_norm"):
        return _exact_residual_norm(s, op.endswith("train"))
    return _exact_product(s, op)
