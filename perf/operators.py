"""Cases of the operators around the optimizer step: activations kept in 8 bits
for the backward pass (store and read back, RMSNorm and SwiGLU forward and
backward over them, the weight gradient of a linear layer from them) and the
clipped policy loss with its gradient.

`run` computes a case in elementary torch operations in 32 bits, or, with
`own` set, by the calls a training loop makes of this package.  `exact` gives
the same outputs from the definitions in 64 bits.

The 8-bit form of an activation x[rows, cols]: one OCP FP8 E4M3 code per
element, every run of 32 consecutive elements of a row with one scale byte b
(value = code * 2^(b - 127)), the smallest exponent >= -127 whose largest
code value, 448, reaches the run's largest magnitude.  Rows are padded with
zeros to whole runs.  Codes are returned as float8_e4m3fn and scales as
float8_e8m0fnu: the values that the bytes stand for.
"""
import math

import torch

own = False

DEVICE = "cuda"
RUN = 32
EPS = 1e-5
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One new row of a residual stream stored and read back: latency alone.
        {"name": "checkpoint_1x4096", "op": "checkpoint", "type": "bf16", "rows": 1, "cols": 4096},
        # A layer's input at full length, stored in the forward pass and read back.
        {"name": "checkpoint_16384x8192", "op": "checkpoint", "type": "bf16", "rows": 16384, "cols": 8192},
        # A decoder layer's norm, one packed batch of 8192 tokens.
        {"name": "norm_8192x4096", "op": "norm", "type": "bf16", "rows": 8192, "cols": 4096},
        # Its backward with the residual stream's gradient, and the norm's output
        # made again in 8 bits for the weight gradients of the projections behind it.
        {"name": "norm_bwd_4096x8192", "op": "norm_bwd", "type": "bf16", "rows": 4096, "cols": 8192},
        # A gated MLP in fp32 at ragged sizes: rows of a short micro-batch.
        {"name": "gate_f32_333x5001", "op": "gate", "type": "f32", "rows": 333, "cols": 5001},
        # The gated MLP's backward at the 8B model's width, its output made again
        # in 8 bits for the down projection's weight gradient.
        {"name": "gate_bwd_8192x14336", "op": "gate_bwd", "type": "bf16", "rows": 8192, "cols": 14336},
        # Weight gradients of an attention projection and of an MLP projection.
        {"name": "wgrad_8192x4096x4096", "op": "wgrad", "type": "bf16", "tokens": 8192, "out": 4096, "cols": 4096},
        {"name": "wgrad_16384x14336x4096", "op": "wgrad", "type": "bf16", "tokens": 16384, "out": 14336, "cols": 4096},
        # fp32 output gradients, ragged in every direction.
        {"name": "wgrad_f32_777x1000x2051", "op": "wgrad", "type": "f32", "tokens": 777, "out": 1000, "cols": 2051},
        # Few answer tokens over the whole vocabulary: the last, short micro-batch.
        {"name": "policy_24x128256", "op": "policy", "type": "bf16", "rows": 24, "cols": 128256},
        # A full micro-batch of answer tokens, a tenth of them prompt or padding.
        {"name": "policy_8192x128256", "op": "policy", "type": "bf16", "rows": 8192, "cols": 128256},
        # fp32 logits of an odd vocabulary.
        {"name": "policy_f32_1000x32003", "op": "policy", "type": "f32", "rows": 1000, "cols": 32003},
    ]


def _size(rng, low, high):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and v >= 128:
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["checkpoint", "norm", "norm_bwd", "gate", "gate_bwd", "wgrad", "policy"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "wgrad":
        c = {"op": op, "type": kind, "tokens": _size(rng, 1, 16384), "out": _size(rng, 8, 14336), "cols": _size(rng, 8, 14336)}
        most = 8192 * 4096 * 4096 if kind == "f32" else 16384 * 14336 * 4096
        c["tokens"] = max(1, min(c["tokens"], most // (c["out"] * c["cols"])))
        return c
    most = {"checkpoint": 16384 * 8192, "norm": 8192 * 4096, "norm_bwd": 4096 * 8192, "gate": 8192 * 14336, "gate_bwd": 8192 * 14336,
            "policy": 8192 * 128256}[op] // (2 if kind == "f32" else 1)
    cols = _size(rng, 1000, 200000) if op == "policy" else _size(rng, 32, 16384)
    rows = _size(rng, 1, 32768)
    return {"op": op, "type": kind, "rows": max(1, min(rows, most // cols)), "cols": cols}


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, cols = case["op"], case["cols"]
    padded = -(-cols // RUN) * RUN
    kept = padded + padded // RUN  # bytes of a row in 8 bits
    if op == "wgrad":
        t, n = case["tokens"], case["out"]
        return {"bytes": t * (n * e + kept) + n * cols * 4, "flops": 2 * t * n * cols}
    rows = case["rows"]
    n = rows * cols
    if op == "checkpoint":
        return {"bytes": 2 * rows * (cols * e + kept), "flops": 4 * n}
    if op == "norm":
        return {"bytes": rows * (2 * cols * e + kept + 4) + cols * 4, "flops": 8 * n}
    if op == "norm_bwd":
        return {"bytes": rows * (3 * cols * e + 2 * kept + 4) + cols * 8, "flops": 16 * n}
    if op == "gate":
        return {"bytes": rows * (3 * cols * e + 2 * kept), "flops": 12 * n}
    if op == "gate_bwd":
        return {"bytes": rows * (3 * cols * e + 3 * kept), "flops": 20 * n}
    return {"bytes": rows * (2 * cols * e + 8 + 16 + 8), "flops": 8 * n}  # policy


# --------------------------------------------------------------- the inputs ---

def _activation(gen, rows, cols, kind):
    """Unit-scale values with a few loud channels, as hidden states have."""
    x = torch.randn(rows, cols, generator=gen, device=DEVICE)
    loud = torch.rand(cols, generator=gen, device=DEVICE) < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(TYPES[kind])


def _bytes(rows, cols):
    padded = -(-cols // RUN) * RUN
    return (torch.empty(rows, padded, dtype=torch.uint8, device=DEVICE),
            torch.empty(rows, padded // RUN, dtype=torch.uint8, device=DEVICE))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, kind, cols = case["op"], case["type"], case["cols"]
    t = TYPES[kind]
    s = {"op": op, "cols": cols}
    if op == "wgrad":
        rows, n = case["tokens"], case["out"]
        s["codes"], s["scales"] = _store(_activation(gen, rows, cols, kind))
        s["dy"] = (torch.randn(rows, n, generator=gen, device=DEVICE) * 1e-2).to(t)
        s["dw"] = torch.empty(n, cols, device=DEVICE)
        s["workspace"] = _workspace("act8_weight_grad_workspace_bytes", rows, n, cols)
        return s
    rows = case["rows"]
    if op == "checkpoint":
        s["x"] = _activation(gen, rows, cols, kind)
        s["codes"], s["scales"] = _bytes(rows, cols)
        s["back"] = torch.empty_like(s["x"])
    elif op in ("norm", "norm_bwd"):
        x = _activation(gen, rows, cols, kind)
        s["weight"] = 1 + 0.1 * torch.randn(cols, generator=gen, device=DEVICE)
        if op == "norm":
            s |= {"x": x, "y": torch.empty_like(x), "rstd": torch.empty(rows, device=DEVICE)}
            s["codes"], s["scales"] = _bytes(rows, cols)
        else:
            s["codes"], s["scales"] = _store(x)
            s["rstd"] = (x.float().square().mean(1) + EPS).rsqrt()
            s["dy"] = (torch.randn(rows, cols, generator=gen, device=DEVICE) * 1e-2).to(t)
            s["dres"] = (torch.randn(rows, cols, generator=gen, device=DEVICE) * 1e-2).to(t)
            s |= {"dx": torch.empty_like(s["dy"]), "dweight": torch.empty(cols, device=DEVICE)}
            s["out_codes"], s["out_scales"] = _bytes(rows, cols)
            s["workspace"] = _workspace("act8_rmsnorm_backward_workspace_bytes", rows, cols)
    elif op in ("gate", "gate_bwd"):
        both = _activation(gen, rows, 2 * cols, kind)  # one projection gives gate and up side by side
        gate, up = both[:, :cols], both[:, cols:]
        if op == "gate":
            s |= {"gate": gate, "up": up, "out": torch.empty(rows, cols, dtype=t, device=DEVICE)}
            s["gate_codes"], s["gate_scales"] = _bytes(rows, cols)
            s["up_codes"], s["up_scales"] = _bytes(rows, cols)
        else:
            s["gate_codes"], s["gate_scales"] = _store(gate)
            s["up_codes"], s["up_scales"] = _store(up)
            s["dout"] = (torch.randn(rows, cols, generator=gen, device=DEVICE) * 1e-2).to(t)
            s["dboth"] = torch.empty(rows, 2 * cols, dtype=t, device=DEVICE)
            s["out_codes"], s["out_scales"] = _bytes(rows, cols)
    else:
        logits = torch.randn(rows, cols, generator=gen, device=DEVICE, dtype=t if kind == "bf16" else None) * 2
        labels = torch.randint(cols, (rows,), generator=gen, device=DEVICE)
        logits[torch.arange(rows, device=DEVICE), labels] += 8  # an answer's tokens were likely ones
        logits[:, cols - cols // 1000:] = -math.inf  # entries that the vocabulary does not use
        labels = labels.clamp(max=cols - cols // 1000 - 1)
        lse = torch.cat([part.double().logsumexp(1) for part in logits.split(512)])
        logp = logits[torch.arange(rows, device=DEVICE), labels].double() - lse
        s["old"] = (logp + 0.2 * torch.randn(rows, generator=gen, device=DEVICE)).float()
        s["ref"] = (logp + 0.4 * torch.randn(rows, generator=gen, device=DEVICE)).float()
        s["adv"] = torch.randn(rows, generator=gen, device=DEVICE)
        s["weight"] = torch.full((rows,), 1.0 / rows, device=DEVICE)
        s["labels"] = torch.where(torch.rand(rows, generator=gen, device=DEVICE) < 0.1, -100, labels)  # prompt and padding
        s |= {"logits": logits, "dlogits": torch.empty_like(logits), "loss": torch.empty(1, device=DEVICE),
              "logp": torch.empty(rows, device=DEVICE), "kl": torch.empty(rows, device=DEVICE)}
        s["workspace"] = _workspace("policy_loss_workspace_bytes", rows, cols)
    return s


def _workspace(name, *sizes):
    """The device scratch that a caller of the package keeps for calls of these sizes."""
    if not own:
        return None
    import mixed_precision_sharded_amd as mps
    return torch.empty(max(1, getattr(mps, name)(*sizes)), dtype=torch.uint8, device=DEVICE)


# ---------------------------------------------------------- the plain forms ---

def _store(x):
    """(codes, scales) of x[rows, cols], as bytes."""
    rows, cols = x.shape
    padded = -(-cols // RUN) * RUN
    runs = torch.nn.functional.pad(x.float(), (0, padded - cols)).view(rows, padded // RUN, RUN)
    mantissa, exponent = torch.frexp(runs.abs().amax(2))  # magnitude = mantissa * 2^exponent, mantissa in [1/2, 1)
    e = torch.where(mantissa == 0, -127, exponent - 9 + (mantissa > 0.875).int()).clamp(min=-127)
    codes = torch.ldexp(runs, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    return codes.view(rows, padded).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales, cols):
    """The fp32 values that the bytes stand for."""
    rows, padded = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(rows, padded // RUN, RUN)
    return torch.ldexp(v, scales.int().unsqueeze(2) - 127).view(rows, padded)[:, :cols]


def _as_values(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _checkpoint(s):
    codes, scales = _store(s["x"])
    return {"back": _values(codes, scales, s["cols"]).to(s["x"].dtype)}


def _norm(s):
    x = s["x"].float()
    rstd = (x.square().mean(1) + EPS).rsqrt()
    y = (x * rstd[:, None] * s["weight"]).to(s["x"].dtype)
    codes, scales = _as_values(*_store(s["x"]))
    return {"y": y, "rstd": rstd, "codes": codes, "scales": scales}


def _norm_bwd(s):
    xhat = _values(s["codes"], s["scales"], s["cols"]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["dres"].float()
    codes, scales = _as_values(*_store(xhat * s["weight"]))
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).sum(0), "codes": codes, "scales": scales}


def _gate(s):
    g = s["gate"].float()
    out = (g * torch.sigmoid(g) * s["up"].float()).to(s["gate"].dtype)
    gc, gs = _as_values(*_store(s["gate"]))
    uc, us = _as_values(*_store(s["up"]))
    return {"out": out, "gate_codes": gc, "gate_scales": gs, "up_codes": uc, "up_scales": us}


def _gate_bwd(s):
    g = _values(s["gate_codes"], s["gate_scales"], s["cols"])
    u = _values(s["up_codes"], s["up_scales"], s["cols"])
    sig = torch.sigmoid(g)
    d = s["dout"].float()
    dgate = d * u * sig * (1 + g * (1 - sig))
    dup = d * g * sig
    codes, scales = _as_values(*_store(g * sig * u))
    return {"dboth": torch.cat([dgate, dup], 1).to(s["dout"].dtype), "codes": codes, "scales": scales}


def _wgrad(s):
    return {"dw": s["dy"].float().t() @ _values(s["codes"], s["scales"], s["cols"])}


def _policy(s):
    x, labels = s["logits"].float(), s["labels"]
    live = labels >= 0
    at = labels.clamp(min=0)[:, None]
    z = x - x.amax(1, keepdim=True)
    p = z.exp()
    total = p.sum(1, dtype=torch.float64)
    # One value a row: in 64 bits, since the clip's border decides which gradient a row gets.
    logp = z.gather(1, at)[:, 0].double() - total.log()
    ratio = (logp - s["old"]).exp()
    adv, w = s["adv"].double(), s["weight"].double()
    plain, clipped = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    diff = s["ref"] - logp
    kl = diff.exp() - diff - 1
    zero = torch.zeros_like(logp)
    loss = torch.where(live, w * (KL * kl - torch.minimum(plain, clipped)), zero).sum()
    slope = torch.where(live, w * (KL * (1 - diff.exp()) - torch.where(plain <= clipped, plain, zero)), zero)
    p *= (-slope / total).float()[:, None]
    p.scatter_add_(1, at, slope.float()[:, None])
    return {"loss": loss.float().view(1), "logp": torch.where(live, logp, zero).float(),
            "kl": torch.where(live, kl, zero).float(), "dlogits": p.to(s["logits"].dtype)}


_PLAIN = {"checkpoint": _checkpoint, "norm": _norm, "norm_bwd": _norm_bwd, "gate": _gate, "gate_bwd": _gate_bwd, "wgrad": _wgrad, "policy": _policy}


# ------------------------------------------------------ the package's calls ---

def _run_own(s):
    import mixed_precision_sharded_amd as mps
    op = s["op"]
    if op == "checkpoint":
        mps.act8_save(s["x"], s["codes"], s["scales"])
        return {"back": mps.act8_load(s["codes"], s["scales"], s["back"])}
    if op == "norm":
        mps.act8_rmsnorm(s["x"], s["weight"], EPS, s["y"], s["rstd"], s["codes"], s["scales"])
        codes, scales = _as_values(s["codes"], s["scales"])
        return {"y": s["y"], "rstd": s["rstd"], "codes": codes, "scales": scales}
    if op == "norm_bwd":
        mps.act8_rmsnorm_backward(s["dy"], s["codes"], s["scales"], s["rstd"], s["weight"], s["dx"], s["dweight"], s["workspace"],
                                  residual_grad=s["dres"], out_codes=s["out_codes"], out_scales=s["out_scales"])
        codes, scales = _as_values(s["out_codes"], s["out_scales"])
        return {"dx": s["dx"], "dweight": s["dweight"], "codes": codes, "scales": scales}
    if op == "gate":
        mps.act8_swiglu(s["gate"], s["up"], s["out"], s["gate_codes"], s["gate_scales"], s["up_codes"], s["up_scales"])
        gc, gs = _as_values(s["gate_codes"], s["gate_scales"])
        uc, us = _as_values(s["up_codes"], s["up_scales"])
        return {"out": s["out"], "gate_codes": gc, "gate_scales": gs, "up_codes": uc, "up_scales": us}
    if op == "gate_bwd":
        cols = s["cols"]
        mps.act8_swiglu_backward(s["dout"], s["gate_codes"], s["gate_scales"], s["up_codes"], s["up_scales"],
                                 s["dboth"][:, :cols], s["dboth"][:, cols:], out_codes=s["out_codes"], out_scales=s["out_scales"])
        codes, scales = _as_values(s["out_codes"], s["out_scales"])
        return {"dboth": s["dboth"], "codes": codes, "scales": scales}
    if op == "wgrad":
        return {"dw": mps.act8_weight_grad(s["dy"], s["codes"], s["scales"], s["dw"], s["workspace"])}
    mps.policy_loss(s["logits"], s["labels"], s["old"], s["adv"], s["weight"], s["loss"], s["workspace"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                    ref_logp=s["ref"], kl_coef=KL, dlogits=s["dlogits"], token_logp=s["logp"], token_kl=s["kl"])
    return {"loss": s["loss"], "logp": s["logp"], "kl": s["kl"], "dlogits": s["dlogits"]}


# ------------------------------------------------- the definitions, 64 bits ---

def _exact_store(x):
    """(code values, scale values, values) of x in float64, rounding by the grid's own steps."""
    rows, cols = x.shape
    padded = -(-cols // RUN) * RUN
    v = torch.zeros(rows, padded, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, -1, RUN)
    most = v.abs().amax(2)
    scale = torch.exp2(torch.floor(torch.log2(most / 448).clamp(min=-127)))
    scale = torch.where(448 * scale < most, 2 * scale, scale)
    scale = torch.where((448 * scale / 2 >= most) & (scale > 2.0 ** -127), scale / 2, scale)[:, :, None]
    c = v / scale
    step = torch.exp2(torch.floor(torch.log2(c.abs().clamp(min=2.0 ** -6))) - 3)
    c = torch.round(c / step) * step
    return c.view(rows, padded), scale[:, :, 0], (c * scale).view(rows, padded)[:, :cols]


def _exact_values(codes, scales, cols):
    """Bytes to float64: sign, exponent and mantissa read from the code."""
    b = torch.arange(256, device=codes.device)
    exponent, mantissa = (b >> 3) & 15, (b & 7).double()
    table = torch.where(exponent == 0, mantissa * 2.0 ** -9, (1 + mantissa / 8) * torch.exp2(exponent.double() - 7))
    table = torch.where(b >= 128, -table, table)
    return (table[codes.int()] * torch.exp2(scales.double() - 127).repeat_interleave(RUN, 1))[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op, cols = s["op"], s["cols"]
    if op == "checkpoint":
        return {"back": _exact_store(s["x"].double())[2]}
    if op == "norm":
        x = s["x"].double()
        rstd = 1 / torch.sqrt((x * x).sum(1) / cols + EPS)
        code, scale, _ = _exact_store(x)
        return {"y": x * s["weight"].double() * rstd[:, None], "rstd": rstd, "codes": code, "scales": scale}
    if op == "norm_bwd":
        x, r = _exact_values(s["codes"], s["scales"], cols), s["rstd"].double()[:, None]
        dy, w = s["dy"].double(), s["weight"].double()
        dot = (dy * w * x).sum(1, keepdim=True) / cols
        code, scale, _ = _exact_store(x * r * w)
        return {"dx": r * dy * w - r * r * r * x * dot + s["dres"].double(), "dweight": (dy * x * r).sum(0), "codes": code, "scales": scale}
    if op == "gate":
        g, u = s["gate"].double(), s["up"].double()
        gc, gs, _ = _exact_store(g)
        uc, us, _ = _exact_store(u)
        return {"out": g * u / (1 + torch.exp(-g)), "gate_codes": gc, "gate_scales": gs, "up_codes": uc, "up_scales": us}
    if op == "gate_bwd":
        g, u = _exact_values(s["gate_codes"], s["gate_scales"], cols), _exact_values(s["up_codes"], s["up_scales"], cols)
        d, t = s["dout"].double(), torch.exp(-g)
        dgate = d * u * (1 + t + g * t) / (1 + t) ** 2
        code, scale, _ = _exact_store(g * u / (1 + t))
        return {"dboth": torch.cat([dgate, d * g / (1 + t)], 1), "codes": code, "scales": scale}
    if op == "wgrad":
        return {"dw": torch.mm(s["dy"].double().t().contiguous(), _exact_values(s["codes"], s["scales"], cols).contiguous())}
    live, at = s["labels"] >= 0, s["labels"].clamp(min=0)
    rows = torch.arange(len(at), device=at.device)
    lse = torch.cat([part.double().logsumexp(1) for part in s["logits"].split(512)])
    logp = s["logits"][rows, at].double() - lse
    adv, w = s["adv"].double(), s["weight"].double()
    r, q = torch.exp(logp - s["old"].double()), torch.exp(s["ref"].double() - logp)
    held = torch.where(adv > 0, r > 1 + CLIP_HIGH, r < 1 - CLIP_LOW)  # the clip's flat side
    gain = torch.where(held, torch.where(adv > 0, 1 + CLIP_HIGH, 1 - CLIP_LOW), r) * adv
    kl = q - (s["ref"].double() - logp) - 1
    slope = w * live * (KL * (1 - q) - torch.where(held, 0.0, r * adv))
    d = torch.empty(s["logits"].shape, dtype=torch.float64, device=at.device)
    for part, l, k, o in zip(s["logits"].split(512), lse.split(512), slope.split(512), d.split(512)):
        torch.mul(torch.exp(part.double() - l[:, None]), -k[:, None], out=o)
    d[rows, at] += slope
    return {"loss": (w * live * (KL * kl - gain)).sum().view(1), "logp": logp * live, "kl": kl * live, "dlogits": d}
