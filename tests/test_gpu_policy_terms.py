"""The policy loss's terms where one of them has no weight: a KL term that is
only watched."""
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
