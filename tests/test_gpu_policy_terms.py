"""The policy loss's terms on their own: a KL term that is only watched, and the
errors of a row's sum and of the gradient where nothing else hides them."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref
from test_gpu_policy import DEV, INF, TYPES, gen, inputs
from train_reference import U

pytestmark = pytest.mark.gpu

# Each kernel: a row per wavefront, a row per block, kept rows of both sizes, blocks that share a row.
KERNELS = [(5, 50), (600, 300), (66, 9001), (70, 20007), (70, 70001), (5, 40000), (24, 50257)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", KERNELS)
def test_a_kl_term_without_a_coefficient_is_only_watched(dtype, rows, vocab):
    """kl_coef 0: the loss and the gradient are those of the call without ref_logp,
    bit for bit, whatever the KL term is; token_kl has it."""
    s = inputs(gen(vocab), rows, vocab, dtype)
    s["labels"][:] = 7
    s["weight"][:], s["adv"][:] = 0.5, 1.0
    s["adv"][1::2] = -1.0
    s["old"] = (torch.log_softmax(s["x"].double(), 1)[:, 7] + 0.1).float()
    s["ref"] = s["old"] + 0.2
    s["x"][0, 7] = -INF                            # no probability left
    s["x"][2, 7], s["old"][2], s["ref"][2] = -2000.0, -2000.0, -1.0  # e^(ref - l) is past fp64
    s["ref"][3] = float("nan")
    out = {}
    for name in ("with", "without"):
        loss, lp, kl = torch.empty(1, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        d = torch.empty(rows, vocab, dtype=dtype, device=DEV)
        ws = torch.empty(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV)
        mps.policy_loss(s["x"], s["labels"], s["old"], s["adv"], s["weight"], loss, ws, ref_logp=s["ref"] if name == "with" else None,
                        kl_coef=0.0, dlogits=d, token_logp=lp, token_kl=kl)
        out[name] = loss, lp, kl, d
    a, b = out["with"], out["without"]
    assert torch.isfinite(a[0]).all() and torch.isfinite(a[3].float()).all()
    for i in (0, 1, 3):
        assert torch.equal(a[i], b[i])
    assert a[1][0] == -INF and a[2][0] == INF and a[2][2] == INF and torch.isnan(a[2][3]) and not b[2].any()
    others = [i for i in range(rows) if i not in (0, 2, 3)]
    want = ref.policy(s["x"][others], s["labels"][others], s["old"][others], s["adv"][others], s["weight"][others], 0.2, 0.2,
                      s["ref"][others], 0.0)["kl"]
    # d is off by the error of l: at most (6 R + 64) u with a range R below 40, as in the tests of the loss.
    assert ((a[2][others].double() - want).abs() <= (6 * 40 + 64) * U * 3).all()


@pytest.mark.parametrize("rows,vocab", KERNELS)
@pytest.mark.parametrize("dtype", TYPES)
def test_a_label_far_below_the_others(dtype, rows, vocab):
    """Every logit 0 but the label's: the sum is a whole number, so l is off by
    fp64's rounding alone, and the loss, -ratio with an advantage and a weight of
    1, by its own rounding to fp32, 2^-24 (a steepness off by 1.3e-8 shows as 8e-7)."""
    far = -60.0 - 4.0 * torch.arange(rows, device=DEV) % 32  # whole numbers of both types; e^l is nothing beside the sum's last bit
    x = torch.zeros(rows, vocab, dtype=dtype, device=DEV)
    labels = (torch.arange(rows, device=DEV) * 13) % vocab
    x[torch.arange(rows, device=DEV), labels] = far.to(dtype)
    logp = far.double() - torch.log(torch.tensor(vocab - 1.0, dtype=torch.float64, device=DEV))
    old = logp.float()
    one, zero = torch.ones(rows, device=DEV), torch.zeros(rows, device=DEV)
    ws = torch.empty(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV)
    loss, lp, kl = torch.empty(1, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    for i in [0, 1, rows // 2, rows - 1]:
        weight = zero.clone()
        weight[i] = 1.0
        mps.policy_loss(x, labels, old, one, weight, loss, ws, token_logp=lp)
        want = -torch.exp(logp[i] - old[i].double())
        assert (loss[0].double() - want).abs() <= 2.0 ** -24 * 1.001, (i, loss.item(), want.item())
        assert (lp[i].double() - logp[i]).abs() <= logp[i].abs() * 2.0 ** -24 * 1.001
    # d = ref - l of about 1: kl within its rounding and fp64's
    mps.policy_loss(x, labels, old, one, one, loss, ws, ref_logp=old + 1, kl_coef=0.1, token_kl=kl)
    d = (old + 1).double() - logp
    want = torch.exp(d) - d - 1
    assert ((kl.double() - want).abs() <= want * 2.0 ** -24 * 1.001).all()


@pytest.mark.parametrize("rows,vocab", KERNELS)
def test_the_gradient_of_unlikely_tokens_has_no_bias(rows, vocab):
    """fp32 logits 60 to 80 below the largest ones: an exponent's rounding has no
    sign, so what remains in the mean of the relative errors is at most the power's
    1 ulp (2^-23), the factor's and the product's rounding (2^-24 each), and the mean of
    the exponents' own: below 2^-24 |d| / sqrt(n) each way, five times over."""
    g = gen(vocab + rows)
    x = torch.zeros(rows, vocab, device=DEV)
    low = torch.rand(rows, vocab, generator=g, device=DEV) < 0.7
    low[:, 0] = False
    x = torch.where(low, torch.empty_like(x).uniform_(-80.0, -60.0, generator=g), x)
    labels = torch.zeros(rows, dtype=torch.int64, device=DEV)
    one = torch.ones(rows, device=DEV)
    l = -torch.log((~low).sum(1).double())  # the unlikely ones' parts are below fp64's last bit
    d, loss = torch.empty_like(x), torch.empty(1, device=DEV)
    ws = torch.empty(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV)
    mps.policy_loss(x, labels, l.float(), one, one, loss, ws, dlogits=d)
    slope = -torch.exp(l - l.float().double())
    want = -slope[:, None] * torch.exp(x.double() + l[:, None])
    rel = (d.double() / want - 1)[low]
    assert (rel.abs() <= 80 * U * 1.5 + 4 * U).all()  # d's product rounded: 80 log2(e) ln 2 u, and as in the bound of the tests of the loss
    assert rel.mean().abs() <= (2 + 1 + 1) * U + 5 * 80 * U / rel.numel() ** 0.5, rel.mean().item()
