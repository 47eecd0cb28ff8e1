"""What linear_cross_entropy promises for every entry of a bf16 g, in bounds that
are relative to the entry (model_reference.head allows for an error relative to the
row), problems that show them, and the form of its arithmetic in 64 bits, with
mistakes that can be planted in it.  Test infrastructure only."""
import torch

UNIT = 2.0 ** -24       # half a step of fp32
BF16_HALF = 2.0 ** -8   # half a step of bf16, relative
# An exponential that stays between the passes keeps its logarithm to base 2 in steps of 2^-10: half a step is 2^-11 ln 2
# of the value, below 2^-11.  What is below 2^-63 of the largest of its stretch may be lost.
KEPT, FLOOR = 2.0 ** -11, 2.0 ** -63


def problem(tokens, vocab, cols, label_gap=0.0, device="cpu", seed=0):
    """bf16 operands whose labels differ from row to row.  The first feature lifts every label's logit by label_gap where all
    rows share one label; of the last eight features only the labels' rows of the weight have any."""
    g = torch.Generator(device=device).manual_seed(seed + tokens * 7 + vocab * 3 + cols)
    hidden = torch.randn(tokens, cols, generator=g, device=device)
    weight = torch.randn(vocab, cols, generator=g, device=device) * (1.5 / cols ** 0.5)
    labels = torch.randperm(vocab, generator=g, device=device)[:tokens]
    if label_gap:
        labels = labels[:1].expand(tokens).contiguous()
        hidden[:, 0] = 1
        weight[:, 0] = 0
        weight[labels[0], 0] = label_gap
    else:
        there = torch.zeros(vocab, 1, device=device)
        there[labels] = 1
        weight[:, -8:] *= there
    c = torch.rand(tokens, generator=g, device=device) + 0.5
    return hidden.bfloat16(), weight.bfloat16(), labels, c


def exact(hidden, weight, labels, c):
    """dict of g, dh, dw in 64 bits and of the largest errors that the promise allows beside the results' last rounding."""
    h, w, c = hidden.double(), weight.double(), c.double()
    (tokens, k), vocab = h.shape, len(w)
    at = torch.arange(tokens, device=h.device), labels
    x = h @ w.t()
    away = x - x.logsumexp(1)[:, None]
    soft = c.abs()[:, None] * torch.exp(away)
    g = c[:, None] * torch.exp(away)
    g[at] -= c
    # k products in fp32 for the logit and for the row's sum, whose 128 terms a stretch are in fp32 as well.
    dl = 2 * (k + 16) * UNIT * (h.abs() @ w.abs().t()).amax(1) + (128 + 8) * UNIT
    # The exponent: a difference of two logits, its product with log2(e), and the part of log2(e) that is left out, 2^-24 of
    # the difference each at the most.
    of_soft = dl[:, None] + 2.0 ** -20 + away.abs() * 2.0 ** -22
    dg = soft * (of_soft + KEPT + BF16_HALF * (1 + of_soft + KEPT)) + c.abs()[:, None] * FLOOR
    # At the label g keeps 16 bits.
    dg[at] = soft[at] * of_soft[at] + g[at].abs() * (2.0 ** -16 + 2.0 ** -20)
    ga = g.abs() + dg
    return {"g": g, "dh": g @ w, "dw": g.t() @ h, "dh_off": dg @ w.abs() + (vocab + 16) * UNIT * (ga @ w.abs()),
            "dw_off": dg.t() @ h.abs() + (tokens + 16) * UNIT * (ga.t() @ h.abs())}


def outside(got, want, off):
    """How many values are farther off than the bound, with the last rounding to got's type."""
    half = BF16_HALF if got.dtype == torch.bfloat16 else UNIT
    return int((~((got.double() - want).abs() <= off + (want.abs() + off) * half)).sum())


def simulate(hidden, weight, labels, c, correction=1.0, kept="log"):
    """(dh, dw): the operator's roundings of g, with its correction at the label (0: forgotten, -1: of the wrong sign), its
    exponentials kept under the largest of 128 as logarithms, or in fp16, or not at all."""
    h, w = hidden.double(), weight.double()
    at = torch.arange(len(h), device=h.device), labels
    x = h @ w.t()
    lse = x.logsumexp(1)
    if kept:
        stretch = torch.nn.functional.pad(x, (0, -x.shape[1] % 128), value=float("-inf")).view(len(x), -1, 128)
        top = stretch.amax(2, keepdim=True)
        if kept == "fp16":
            e = torch.exp(stretch - top).half().double()
        else:
            steps = ((top - stretch) * (1024 / torch.log(torch.tensor(2.0)).double())).round().clamp(max=65535)
            e = torch.where(steps == 65535, 0.0, torch.exp2(-steps / 1024))
        soft = (e * torch.exp(top - lse[:, None, None])).view(len(x), -1)[:, :x.shape[1]]
    else:
        soft = torch.exp(x - lse[:, None])
    g = c.double()[:, None] * soft
    g[at] = c.double() * (torch.exp(x[at] - lse) - 1)
    rounded = g.bfloat16().double()
    lost = torch.zeros_like(g)
    lost[at] = correction * (g[at] - rounded[at])
    return ((rounded + lost) @ w).bfloat16(), ((rounded + lost.bfloat16().double()).t() @ h).float()
