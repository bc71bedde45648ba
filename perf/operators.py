"""The operators of a selective block, as they are measured: the short causal convolution,
the selective scan and layer norm, each as it is called for prompts, for single tokens and
for training.

`run` computes them in elementary torch operations (32 bits, rounded once at the end) where
`own` is false, and calls the package's entry points where it is true; `exact` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decoded token through the convolution of a 768-wide block (expand 2), batch 1:
        # latency of the call.
        dict(name="conv_step_b1_c1536", op="conv_step", batch=1, chan=1536, width=4, dtype="bf16"),
        # Batched prompts, x half of an in-projection's output (rows of twice the width).
        dict(name="conv_prompt_b8_L4096_c2048", op="conv_prompt", batch=8, len=4096, chan=2048, width=4,
             dtype="bf16", split=True, ragged=False, state=True),
        # A training step on a ragged float32 batch, odd channel count, three taps.
        dict(name="conv_train_ragged_b5_L1999_c777_f32", op="conv_train", batch=5, len=1999, chan=777, width=3,
             dtype="f32", split=False, ragged=True, state=True),
        # One decoded token through the scan, batch 1: latency of the call.
        dict(name="scan_step_b1_c1536", op="scan_step", batch=1, chan=1536, dstate=16, groups=1, dtype="bf16"),
        # One token for each of 256 streams: the states' traffic.
        dict(name="scan_step_b256_c2048", op="scan_step", batch=256, chan=2048, dstate=16, groups=1, dtype="bf16"),
        # An ordinary prompt at batch 1 (one 2048-token segment), few channels to spread.
        dict(name="scan_prompt_b1_L2048_c1536", op="scan_prompt", batch=1, len=2048, chan=1536, dstate=16, groups=1,
             dtype="bf16", split=True, ragged=False, state=True),
        # A long prompt at batch 1.
        dict(name="scan_prompt_b1_L32768_c2048", op="scan_prompt", batch=1, len=32768, chan=2048, dstate=16,
             groups=1, dtype="bf16", split=True, ragged=False, state=False),
        # A ragged float32 batch with odd sizes, two groups and a larger state.
        dict(name="scan_prompt_ragged_b6_L1501_c1110_n32_f32", op="scan_prompt", batch=6, len=1501, chan=1110,
             dstate=32, groups=2, dtype="f32", split=False, ragged=True, state=True),
        # A training step: forward with what its backward needs, then every gradient.
        dict(name="scan_train_b2_L4096_c2048", op="scan_train", batch=2, len=4096, chan=2048, dstate=16, groups=1,
             dtype="bf16", split=True, ragged=False, state=False),
        # One decoded token's norm: latency of the call.
        dict(name="norm_prompt_r1_d768", op="norm_prompt", rows=1, chan=768, dtype="bf16"),
        # A training step over a batch of 8 x 4096 tokens.
        dict(name="norm_train_r32768_d2048", op="norm_train", rows=32768, chan=2048, dtype="bf16"),
        # A training step in float32 with an odd width and an odd number of rows.
        dict(name="norm_train_r4099_d1025_f32", op="norm_train", rows=4099, chan=1025, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_prompt", "conv_train", "scan_step", "scan_prompt", "scan_prompt",
                     "scan_train", "norm_prompt", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        chan = _spread(rng, 64, 8192)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(65536, (1 << 25) // chan))), chan=chan, dtype=dtype)
    groups = rng.choice([1, 1, 2])
    chan = groups * (_spread(rng, 64, 4096) // groups)
    if rng.random() < 0.5:                       # half of the cases at a multiple of 64, as most widths are
        chan = 64 * groups * max(1, chan // (64 * groups))
    c = dict(op=op, chan=chan, dtype=dtype)
    if op.startswith("conv"):
        c["width"] = rng.choice([2, 3, 4, 4])
    else:
        c["dstate"] = rng.choice([16, 16, 16, 32, 64])
        c["groups"] = groups
    if op.endswith("step"):
        c["batch"] = _spread(rng, 1, 256)
        return c
    c["batch"] = _spread(rng, 1, 16)
    room = (1 << 25) if op.startswith("conv") else (1 << 28) // c["dstate"] if op == "scan_train" else (1 << 29) // c["dstate"]
    c["len"] = _spread(rng, 1, max(1, min(32768, room // (c["batch"] * chan))))
    c["split"] = rng.random() < 0.5
    c["ragged"] = rng.random() < 0.4
    c["state"] = rng.random() < 0.5
    return c


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    ch = case["chan"]
    if op.startswith("norm"):
        n = case["rows"] * ch
        if op == "norm_prompt":
            return {"bytes": 2 * n * e + 8 * ch, "flops": 8 * n}
        # x in, y out; dy in, dx out (x and the statistics are what the step has at hand)
        return {"bytes": 4 * n * e + 16 * ch + 8 * case["rows"], "flops": 8 * n + 14 * n}
    b, length = case["batch"], case.get("len", 1)
    n = b * length * ch
    if op.startswith("conv"):
        w = case["width"]
        state = 2 * b * (w - 1) * ch * e
        par = 4 * ch * (w + 1)
        if op == "conv_train":
            return {"bytes": 4 * n * e + state + 2 * par, "flops": n * (2 * w + 6) + n * (6 * w + 12)}
        return {"bytes": 2 * n * e + state + par, "flops": n * (2 * w + 6)}
    nst = case["dstate"]
    par = 4 * ch * (nst + 2)
    bc = 2 * b * length * case["groups"] * nst * e
    state = 2 * b * ch * nst * 4
    if op == "scan_train":
        # u, delta, z, dout in; y, du, ddelta, dz out; B, C in, their gradients out
        return {"bytes": 8 * n * e + 2 * bc + 2 * par + state // 2, "flops": n * (8 * nst + 16) + n * (19 * nst + 40)}
    return {"bytes": 4 * n * e + bc + par + state, "flops": n * (8 * nst + 16)}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op, ch = case["op"], case["chan"]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if op.startswith("norm"):
        s["x"] = randn(case["rows"], ch, std=2.0) + 0.5
        s["weight"] = 1.0 + 0.2 * randn(ch, dtype=torch.float32)
        s["bias"] = 0.1 * randn(ch, dtype=torch.float32)
        if op == "norm_train":
            s["dy"] = randn(case["rows"], ch)
        return s
    b, length = case["batch"], case.get("len", 1)
    step = op.endswith("step")
    lead = (b,) if step else (b, length)
    # the two halves of an in-projection's output are views with rows of twice the width
    x = randn(*lead, 2 * ch) if case.get("split") else randn(*lead, ch)
    x, z = (x[..., :ch], x[..., ch:]) if case.get("split") else (x, None)
    s["lengths"] = None
    if case.get("ragged"):
        s["lengths"] = (rand(b) * (length + 1)).to(torch.int32)
        s["lengths"][0] = length
        if b > 2:
            s["lengths"][1] = 0                      # a row with nothing in it
    if op.startswith("conv"):
        w = case["width"]
        s["x"] = x
        s["weight"] = randn(ch, w, std=1.0 / math.sqrt(w), dtype=torch.float32)
        s["bias"] = randn(ch, std=0.1, dtype=torch.float32)
        s["state"] = randn(b, w - 1, ch) if step or case["state"] else None
        if step:
            s["state_out"] = torch.empty_like(s["state"])
        if op == "conv_train":
            s["dy"] = randn(b, length, ch)
        return s
    n, g = case["dstate"], case["groups"]
    s["u"] = x
    s["z"] = randn(*lead, ch) if z is None else z
    s["delta"] = randn(*lead, ch, std=0.5)
    # step sizes spread over [1e-3, 0.1] through the bias, decay rates 1..N as a layer starts with
    step0 = torch.exp(rand(ch) * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = step0 + torch.log(-torch.expm1(-step0))
    s["A"] = -(torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * randn(ch, n, dtype=torch.float32)))
    s["D"] = rand(ch)
    if case.get("split"):
        bc = randn(*lead, 48 + 2 * g * n)            # behind the low-rank step sizes in one projection's output
        s["B"] = bc[..., 48:48 + g * n].unflatten(-1, (g, n))
        s["C"] = bc[..., 48 + g * n:].unflatten(-1, (g, n))
    else:
        s["B"], s["C"] = randn(*lead, g, n), randn(*lead, g, n)
    s["state"] = randn(b, ch, n, std=0.3, dtype=torch.float32) if step or case["state"] else None
    if step:
        s["state_out"] = torch.empty_like(s["state"])
    if op == "scan_train":
        s["dy"] = randn(b, length, ch)
    return s


# ---------------------------------------------------------------------- the plain forms
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _dsilu(v):
    sig = 1.0 / (1.0 + torch.exp(-v))
    return sig * (1.0 + v * (1.0 - sig))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _inside(lengths, length):
    """[b, L, 1]: the tokens of each row."""
    return (torch.arange(length, device=lengths.device)[None, :] < lengths[:, None])[..., None]


def _plain_conv(s, train):
    x, w = s["x"].float(), s["weight"]
    b, length, ch = x.shape
    k = w.shape[1]
    lengths = s["lengths"]
    if lengths is not None:
        inside = _inside(lengths, length)
        x = torch.where(inside, x, torch.zeros_like(x))
    head = s["state"].float() if s["state"] is not None else x.new_zeros(b, k - 1, ch)
    full = torch.cat([head, x], 1)                           # token t is at t + k - 1
    pre = s["bias"] + sum(full[:, j:j + length] * w[:, j] for j in range(k))
    y = _silu(pre)
    if lengths is not None:
        y = torch.where(inside, y, torch.zeros_like(y))
        at = lengths[:, None].long() + torch.arange(k - 1, device=x.device)[None, :]
        last = torch.gather(full, 1, at[..., None].expand(b, k - 1, ch))
    else:
        last = full[:, length:]
    out = (y.to(s["x"].dtype), last.to(s["x"].dtype))
    if not train:
        return out
    dpre = s["dy"].float() * _dsilu(pre)
    if lengths is not None:
        dpre = torch.where(inside, dpre, torch.zeros_like(dpre))
    dfull = torch.zeros_like(full)
    for j in range(k):
        dfull[:, j:j + length] += dpre * w[:, j]
    dw = torch.stack([(dpre * full[:, j:j + length]).sum((0, 1)) for j in range(k)], 1)
    dinit = dfull[:, :k - 1].to(s["x"].dtype) if s["state"] is not None else None
    return out + (dfull[:, k - 1:].to(s["x"].dtype), dw, dpre.sum((0, 1))) + (() if dinit is None else (dinit,))


def _plain_conv_step(s):
    full = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    pre = s["bias"] + (full * s["weight"].t()).sum(1)
    return _silu(pre).to(s["x"].dtype), full[:, 1:].to(s["x"].dtype)


def _plain_scan(s, train):
    """Chunks side by side: each chunk's end state from nothing, the states passed from
    chunk to chunk, and each chunk once more from the state that enters it."""
    u, delta, z = s["u"].float(), s["delta"].float(), s["z"].float()
    b, length, ch = u.shape
    A = s["A"]
    n = A.shape[1]
    per = ch // s["B"].shape[2]
    lengths = s["lengths"]
    raw = delta + s["delta_bias"]
    dt = _softplus(raw)
    Bm, Cm = s["B"].float(), s["C"].float()
    if lengths is not None:
        inside = _inside(lengths, length)
        dt = torch.where(inside, dt, torch.zeros_like(dt))
        u = torch.where(inside, u, torch.zeros_like(u))
        Bm = torch.where(inside[..., None], Bm, torch.zeros_like(Bm))
        Cm = torch.where(inside[..., None], Cm, torch.zeros_like(Cm))
    q = max(1, min(128, length, 1 << max(4, int(math.log2(length)) // 2 + 1)))
    nc = -(-length // q)

    def chunks(t):
        pad = t.new_zeros(b, nc * q - length, *t.shape[2:])
        return torch.cat([t, pad], 1).reshape(b, nc, q, *t.shape[2:])

    dtc, uc, Bc, Cc = chunks(dt), chunks(u), chunks(Bm), chunks(Cm)
    decay = torch.exp(dtc.sum(2)[..., None] * A)             # [b, nc, ch, n]

    def spread(t):                                           # groups to their channels
        return t.repeat_interleave(per, 2) if t.shape[2] > 1 else t

    def through(h, keep):
        ys, hs, before = [], [], []
        for i in range(q):
            a = torch.exp(dtc[:, :, i, :, None] * A)
            if train and keep:
                before.append(a * h)
            h = a * h + (dtc[:, :, i] * uc[:, :, i])[..., None] * spread(Bc[:, :, i])
            if keep:
                ys.append((h * spread(Cc[:, :, i])).sum(-1))
                if train:
                    hs.append(h)
        return h, ys, hs, before

    h = s["state"] if s["state"] is not None else u.new_zeros(b, ch, n)
    end = through(u.new_zeros(b, nc, ch, n), False)[0]
    entry = []
    for c in range(nc):
        entry.append(h)
        h = decay[:, c] * h + end[:, c]
    last = h
    _, ys, hs, before = through(torch.stack(entry, 1), True)
    y = torch.stack(ys, 2).reshape(b, nc * q, ch)[:, :length] + s["D"] * u
    out = y * _silu(z)
    if lengths is not None:
        out = torch.where(inside, out, torch.zeros_like(out))
    act = s["u"].dtype
    if not train:
        return out.to(act), last
    dy = s["dy"].float()
    r, dz = dy * _silu(z), dy * y * _dsilu(z)
    if lengths is not None:
        r, dz = torch.where(inside, r, torch.zeros_like(r)), torch.where(inside, dz, torch.zeros_like(dz))
    rc = chunks(r)

    def back(carry, keep):
        """carry: a_t g_t of the token after the chunk."""
        dq, dd = [None] * q, [None] * q
        dB, dC = [None] * q, [None] * q
        dA = 0.0
        for i in reversed(range(q)):
            g = rc[:, :, i, :, None] * spread(Cc[:, :, i]) + carry
            if keep:
                dq[i] = (g * spread(Bc[:, :, i])).sum(-1)
                gp = g * before[i]
                dd[i] = (gp * A).sum(-1)
                dA = dA + (gp * dtc[:, :, i, :, None]).sum((0, 1))
                x = (dtc[:, :, i] * uc[:, :, i])[..., None]
                dB[i] = (g * x).unflatten(2, (-1, per)).sum(3)
                dC[i] = (rc[:, :, i, :, None] * hs[i]).unflatten(2, (-1, per)).sum(3)
            carry = torch.exp(dtc[:, :, i, :, None] * A) * g
        return carry, dq, dd, dA, dB, dC

    start = back(u.new_zeros(b, nc, ch, n), False)[0]
    carry = u.new_zeros(b, ch, n)
    into = [None] * nc
    for c in reversed(range(nc)):
        into[c] = carry
        carry = decay[:, c] * carry + start[:, c]
    dinit = carry
    _, dq, dd, dA, dB, dC = back(torch.stack(into, 1), True)

    def whole(ts):
        t = torch.stack(ts, 2)
        return t.reshape(b, nc * q, *t.shape[3:])[:, :length]

    dq, dd = whole(dq), whole(dd)
    ddelta = (dd + dq * u) / (1.0 + torch.exp(-raw))
    du = dq * dt + s["D"] * r
    if lengths is not None:
        ddelta, du = torch.where(inside, ddelta, torch.zeros_like(ddelta)), torch.where(inside, du, torch.zeros_like(du))
    grads = (du.to(act), ddelta.to(act), dA, whole(dB).to(act), whole(dC).to(act), (r * u).sum((0, 1)), dz.to(act),
             ddelta.sum((0, 1)))
    return (out.to(act), last) + grads + (() if s["state"] is None else (dinit,))


def _plain_scan_step(s):
    u, z = s["u"].float(), s["z"].float()
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    per = u.shape[1] // s["B"].shape[1]
    Bm, Cm = s["B"].float().repeat_interleave(per, 1), s["C"].float().repeat_interleave(per, 1)
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * u)[..., None] * Bm
    y = (h * Cm).sum(-1) + s["D"] * u
    return (y * _silu(z)).to(s["u"].dtype), h


def _plain_norm(s, train):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + _EPS)
    hat = xc * rstd
    y = (hat * s["weight"] + s["bias"]).to(s["x"].dtype)
    if not train:
        return y
    dy = s["dy"].float()
    gw = dy * s["weight"]
    dx = rstd * (gw - gw.mean(1, keepdim=True) - hat * (gw * hat).mean(1, keepdim=True))
    return y, dx.to(s["x"].dtype), (dy * hat).sum(0), dy.sum(0)


# ------------------------------------------------------------------------------ a pass
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"conv_step": lambda: _plain_conv_step(s), "conv_prompt": lambda: _plain_conv(s, False),
                "conv_train": lambda: _plain_conv(s, True), "scan_step": lambda: _plain_scan_step(s),
                "scan_prompt": lambda: _plain_scan(s, False), "scan_train": lambda: _plain_scan(s, True),
                "norm_prompt": lambda: _plain_norm(s, False), "norm_train": lambda: _plain_norm(s, True)}[op]()
    from chunked_linear_recurrence_amd import ssd
    if op == "conv_step":
        y = ssd.conv_step(s["x"], s["weight"], s["bias"], s["state"], state_out=s["state_out"])
        return y, s["state_out"]
    if op.startswith("conv"):
        y, last = ssd.conv_fwd(s["x"], s["weight"], s["bias"], s["state"], lengths=s["lengths"])
        if op == "conv_prompt":
            return y, last
        g = ssd.conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["state"], lengths=s["lengths"])
        return (y, last, g.dx, g.dweight, g.dbias) + (() if s["state"] is None else (g.dinit,))
    if op == "scan_step":
        y = ssd.selective_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                               s["state"], state_out=s["state_out"])
        return y, s["state_out"]
    if op == "scan_prompt":
        return ssd.selective_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                                 s["state"], lengths=s["lengths"])
    if op == "scan_train":
        y, last, kept = ssd.selective_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                          s["delta_bias"], s["state"], lengths=s["lengths"], keep=True)
        g = ssd.selective_bwd(s["dy"], s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                              kept, lengths=s["lengths"])
        return ((y, last, g.du, g.ddelta, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddelta_bias) +
                (() if s["state"] is None else (g.dinit,)))
    if op == "norm_prompt":
        return ssd.norm_fwd(s["x"], s["weight"], s["bias"], _EPS)
    y, mean, rstd = ssd.norm_fwd(s["x"], s["weight"], s["bias"], _EPS, want_stats=True)
    g = ssd.norm_bwd(s["dy"], s["x"], s["weight"], mean, rstd)
    return y, g.dx, g.dweight, g.dbias


# ------------------------------------------------------------------- the definitions, 64 bits
def _exact_conv(s, op):
    """Row by row and tap by tap over each row's own tokens; gradients by differentiation."""
    x = s["x"].double()
    x = x[:, None] if op == "conv_step" else x
    b, length, ch = x.shape
    k = s["weight"].shape[1]
    w, bias = s["weight"].double(), s["bias"].double()
    init = s["state"].double() if s["state"] is not None else None
    train = op == "conv_train"
    leaves = [x, w, bias] + ([init] if init is not None else [])
    if train:
        for t in leaves:
            t.requires_grad_(True)
    lens = [length] * b if s["lengths"] is None else s["lengths"].tolist()
    ys, lasts = [], []
    with torch.set_grad_enabled(train):
        for i in range(b):
            m = lens[i]
            head = init[i] if init is not None else x.new_zeros(k - 1, ch)
            row = torch.cat([head, x[i, :m]], 0)
            y = torch.nn.functional.silu(bias + sum(row[j:j + m] * w[:, j] for j in range(k)))
            ys.append(torch.cat([y, x.new_zeros(length - m, ch)], 0))
            lasts.append(row[m:])
        y = torch.stack(ys)
        if train:
            grads = torch.autograd.grad((y * s["dy"].double()).sum(), leaves, allow_unused=True)
            grads = tuple(torch.zeros_like(t) if g is None else g for g, t in zip(grads, leaves))
    y, last = y.detach(), torch.stack(lasts).detach()
    if op == "conv_step":
        return y[:, 0], last
    return (y, last) + (grads if train else ())


def _exact_scan(s, op):
    """Token by token; gradients by differentiation."""
    act = [s[k].double() for k in ("u", "delta", "B", "C", "z")]
    if op == "scan_step":
        act = [t[:, None] for t in act]
    par = [s[k].double() for k in ("A", "D", "delta_bias")]
    h = s["state"].double() if s["state"] is not None else None
    train = op == "scan_train"
    leaves = act + par + ([h] if h is not None else [])
    if train:
        for t in leaves:
            t.requires_grad_(True)
    u, delta, Bm, Cm, z = act
    A, D, bias = par
    b, length, ch = u.shape
    grp = torch.arange(ch, device=u.device) // (ch // Bm.shape[2])
    if h is None:
        h = u.new_zeros(b, ch, A.shape[1])
    ys = [] if train else u.new_empty(b, length, ch)
    with torch.set_grad_enabled(train):
        dt = torch.logaddexp(delta + bias, torch.zeros((), dtype=torch.float64, device=u.device))
        x = dt * u
        for t in range(length):
            new = torch.exp(dt[:, t, :, None] * A) * h + x[:, t, :, None] * Bm[:, t][:, grp]
            if s["lengths"] is not None:
                new = torch.where((t < s["lengths"])[:, None, None], new, h)
            h = new
            y = (h * Cm[:, t][:, grp]).sum(-1)
            if train:
                ys.append(y)
            else:
                ys[:, t] = y
        y = torch.stack(ys, 1) if train else ys
        y = (y + D * u) * torch.nn.functional.silu(z)
        if s["lengths"] is not None:
            y = y * (torch.arange(length, device=u.device)[None, :, None] < s["lengths"][:, None, None])
        if train:
            g = torch.autograd.grad((y * s["dy"].double()).sum(), leaves)
    y, h = y.detach(), h.detach()
    if op == "scan_step":
        return y[:, 0], h
    if op == "scan_prompt":
        return y, h
    du, ddelta, dB, dC, dz, dA, dD, dbias = g[:8]
    return (y, h, du, ddelta, dA, dB, dC, dD, dz, dbias) + tuple(g[8:])


def exact(case, seed):
    op = case["op"]
    if op == "scan_train" and case["batch"] * case["len"] * case["chan"] * case["dstate"] > 1 << 28:
        return None                                  # the differentiated loop would not fit beside the rest
    s = prepare(case, seed)
    if op.startswith("conv"):
        return _exact_conv(s, op)
    if op.startswith("scan"):
        return _exact_scan(s, op)
    x, w, bias = s["x"].double(), s["weight"].double(), s["bias"].double()
    train = op == "norm_train"
    if train:
        for t in (x, w, bias):
            t.requires_grad_(True)
    with torch.set_grad_enabled(train):
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        y = (x - mean) / torch.sqrt(var + _EPS) * w + bias
        if not train:
            return y
        dx, dw, db = torch.autograd.grad((y * s["dy"].double()).sum(), (x, w, bias))
    return y.detach(), dx, dw, db
