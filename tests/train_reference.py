"""Plain 64-bit forms of the operators of include/mps_train.h, for the tests:
written from the header's formulas with torch in float64, on any device.
The 8-bit rule itself comes from the oracle (`keep`)."""
import numpy as np
import torch

RUN = 32
U = 2.0 ** -24  # unit roundoff of fp32


def half_step(dtype) -> float:
    """Largest relative error of one rounding to this type."""
    return torch.finfo(dtype).eps / 2


def row_of(cols: int) -> int:
    return (cols + RUN - 1) // RUN * RUN


def keep(oracle_lib, x: torch.Tensor):
    """(codes, scales) of a matrix as uint8 tensors on the CPU, row by row by the oracle."""
    rows, cols = x.shape
    padded = np.zeros((rows, row_of(cols)), np.float32)
    padded[:, :cols] = x.detach().float().cpu().numpy()
    if not rows:
        return torch.zeros(0, row_of(cols), dtype=torch.uint8), torch.zeros(0, row_of(cols) // RUN, dtype=torch.uint8)
    codes, scales = oracle_lib.quantize(padded.reshape(-1), 0)
    return (torch.from_numpy(np.asarray(codes).reshape(rows, -1).copy()),
            torch.from_numpy(np.asarray(scales).reshape(rows, -1).copy()))


def values(codes: torch.Tensor, scales: torch.Tensor, cols: int) -> torch.Tensor:
    """float64 values of codes and scales, decoded bit by bit, on their device."""
    b = torch.arange(256, dtype=torch.float64)
    e, m = ((b % 128) / 8).floor(), b % 8
    table = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7.0)) * torch.where(b >= 128, -1.0, 1.0)
    table[127], table[255] = float("nan"), float("nan")
    scale = torch.exp2(b - 127)
    scale[255] = float("nan")
    v = table.to(codes.device)[codes.long()] * scale.to(codes.device)[scales.long()].repeat_interleave(RUN, 1)
    return v[:, :cols]


def rmsnorm(x, weight, eps):
    r = 1 / torch.sqrt((x * x).mean(1) + eps)
    return x * r[:, None] * weight, r


def rmsnorm_backward(dy, x, r, weight, residual=None):
    """dx, dweight and the norm's output of the kept x."""
    xh = x * r[:, None]
    g = dy * weight
    dx = r[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    return dx if residual is None else dx + residual, (dy * xh).sum(0), xh * weight


def swiglu(g, u):
    return g * u / (1 + torch.exp(-g))


def swiglu_backward(d, g, u):
    s = 1 / (1 + torch.exp(-g))
    return d * u * s * (1 + g * (1 - s)), d * g * s


def policy(logits, labels, old, adv, weight, low, high, ref=None, kl_coef=0.0):
    """A dict of loss, logp, kl, slope and dlogits, all float64."""
    x = logits.double()
    rows, vocab = x.shape
    live = (labels >= 0) & (labels < vocab) & (weight != 0) & ~(x == -float("inf")).all(1)
    at = labels.clamp(0, vocab - 1)[:, None]
    top = x.amax(1, keepdim=True)
    x = x - torch.where(top == -float("inf"), torch.zeros_like(top), top)  # exact, or far below the sum
    lse = torch.logsumexp(x, 1)
    zero = torch.zeros(rows, dtype=torch.float64, device=x.device)
    logp = torch.where(live, x.gather(1, at)[:, 0] - lse, zero)
    a, w, o = adv.double(), weight.double(), old.double()
    ratio = torch.exp(logp - o)
    plain, held = ratio * a, ratio.clamp(1 - low, 1 + high) * a
    flat = plain > held
    gain = torch.where(a == 0, zero, torch.where(flat, held, plain))
    slope = torch.where((a == 0) | flat, zero, -plain)
    kl = zero
    if ref is not None:
        d = ref.double() - logp
        kl = torch.exp(d) - d - 1
        gain, slope = gain - kl_coef * kl, slope + kl_coef * (1 - torch.exp(d))
    kl = torch.where(live, kl, zero)
    slope = torch.where(live, slope * w, zero)
    loss = torch.where(live, -w * gain, zero)
    p = torch.exp(x - lse[:, None])
    d = torch.where(live[:, None], -slope[:, None] * p, torch.zeros_like(x))
    d[torch.arange(rows, device=x.device), at[:, 0]] += slope
    return {"loss": loss.sum(), "row_loss": loss, "logp": logp, "kl": kl, "slope": slope, "dlogits": d, "live": live,
            "p": torch.where(live[:, None], p, torch.zeros_like(p))}
