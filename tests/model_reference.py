"""The operators of include/mps_model.h in 64 bits, from their formulas, and the
bounds that their own roundings allow.  Test infrastructure only."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


# ------------------------------------------------------------- embedding ---

def embedding(ids, table, scale):
    known = (ids >= 0) & (ids < len(table))
    out = table.double()[ids.clamp(0, len(table) - 1)] * float(np.float32(scale))
    return torch.where(known[:, None], out, 0.0)


def embedding_grad(dout, ids, vocab, scale):
    """(gradient, the sum of the magnitudes that went into it, tokens of each row)."""
    known = ((ids >= 0) & (ids < vocab)).nonzero()[:, 0]
    d = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device)
    size, count = d.clone(), torch.zeros(vocab, dtype=torch.float64, device=dout.device)
    d.index_add_(0, ids[known], dout[known].double())
    size.index_add_(0, ids[known], dout[known].double().abs())
    count.index_add_(0, ids[known], torch.ones_like(known, dtype=torch.float64))
    s = float(np.float32(scale))
    return d * s, size * abs(s), count


# --------------------------------------------------------------- dropout ---

def philox(counter, key):
    """Philox4x32-10 on Python integers: counter of four words, key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(rows, cols, seed, site, step):
    """The 16 bits of every element, int64 [rows, cols]; numpy's 64-bit words."""
    units = -(-cols // 8)
    at = np.arange(rows * units, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    c = [at & m, at >> s, np.full_like(at, site), np.full_like(at, step & 0xFFFFFFFF)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k0), b & m, (a >> s) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    halves = np.stack([w for word in c for w in (word & np.uint64(0xFFFF), word >> np.uint64(16))], 1)
    return torch.from_numpy(halves.reshape(rows, units * 8)[:, :cols].astype(np.int64))


def dropout(x, p, seed, site, step, residual=None):
    """The bits that the operator gives: each fp32 operation rounds once, then the type."""
    threshold = round(p * 65536)
    scale = 0.0 if threshold == 65536 else np.float32(65536 / (65536 - threshold))
    keep = (draws(*x.shape, seed, site, step) >= threshold).to(x.device)
    y = torch.where(keep, x.float() * float(scale), 0.0)
    return (y if residual is None else residual.float() + y).to(x.dtype)


# ---------------------------------------------------------- the head's loss ---

def live_rows(labels, token_weight, vocab):
    live = (labels >= 0) & (labels < vocab)
    return live if token_weight is None else live & (token_weight != 0)


def head(hidden, weight, labels, token_weight):
    """dict of loss, logp, dh, dw in 64 bits, and beside each the largest error that
    the operator's roundings allow (its own type's last rounding apart)."""
    dtype, (tokens, k), vocab = hidden.dtype, hidden.shape, len(weight)
    live = live_rows(labels, token_weight, vocab).nonzero()[:, 0]
    h, w, at = hidden[live].double(), weight.double(), labels[live]
    c = token_weight[live].double()
    index = torch.arange(len(live), device=h.device)
    x = h @ w.t()
    size = h.abs() @ w.abs().t()
    # A logit: k exact products summed in fp32 in some order, and with fp32 operands what six products of parts leave out
    # (parts of at most 2^-7 and 2^-15 of a value: 2 * 2^-22 + 2^-30).
    unit = 2.0 ** -24
    per = (k + 16) * unit + (2.0 ** -21 + 2.0 ** -30 if dtype == torch.float32 else 0.0)
    dx = per * size.amax(1) if vocab else size.sum(1)
    lse = x.logsumexp(1)
    logp = x[index, at] - lse
    # Exponentials within 2^-21, sums of 128 of them in fp32.
    dl = 2 * dx + (128 + 8) * unit
    g = c[:, None] * torch.exp(x - lse[:, None])
    g[index, at] -= c
    # g: its logit's and sum's errors act on the softmax, then one rounding to the operands' type (three parts hold the 24
    # bits of an fp32 value).
    soft = c.abs()[:, None] * torch.exp(x - lse[:, None])
    # With bf16 operands the exponentials that stay from the first pass are kept in 16 bits on the way: 2^-11 of each, and
    # for what is smaller than they reach far more than they lose (head_precision has the bounds that are relative to each).
    half = soft * 2.0 ** -11 + c.abs()[:, None] * 2.0 ** -25 if dtype == torch.bfloat16 else 0.0
    dg = half + soft * (dl[:, None] + 2.0 ** -20) + (g.abs() + soft * dl[:, None]) * HALF[dtype] + c.abs()[:, None] * 2 ** -22 * (soft > 0)
    ga = g.abs() + dg
    more = 2.0 ** -21 + 2.0 ** -30 if dtype == torch.float32 else 0.0
    full = lambda v, n: torch.zeros(n, *v.shape[1:], dtype=torch.float64, device=v.device).index_copy_(0, live, v)  # noqa: E731
    dh_off = dg @ w.abs() + ((vocab + 16) * unit + more) * (ga @ w.abs())
    dw_off = dg.t() @ h.abs() + ((tokens + 16) * unit + more) * (ga.t() @ h.abs())
    return {"loss": -(c * logp).sum(), "loss_off": (c.abs() * dl).sum(), "logp": full(logp, tokens), "logp_off": full(dl, tokens),
            "dh": full(g @ w, tokens), "dh_off": full(dh_off, tokens), "dw": g.t() @ h, "dw_off": dw_off}
