"""linear_cross_entropy's bf16 g, entry by entry, against the bounds of
head_precision: relative to the entry, not to its row."""
import pytest
import torch

import head_precision as hp
import mixed_precision_sharded_amd as mps

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def gradients(hidden, weight, labels, c, dw_type):
    (tokens, cols), vocab = hidden.shape, len(weight)
    ws = torch.empty(mps.linear_cross_entropy_workspace_bytes(tokens, vocab, cols, BF16), dtype=torch.uint8, device=DEV).fill_(255)
    loss, dh = torch.empty(1, device=DEV), torch.empty_like(hidden)
    dw = torch.empty(vocab, cols, dtype=dw_type, device=DEV)
    mps.linear_cross_entropy(hidden, weight, labels, c, loss, ws, dhidden=dh, dweight=dw)
    return dh, dw


@pytest.mark.parametrize("gap", [12.0, 18.0, 24.0, 34.0])
@pytest.mark.parametrize("tokens,vocab,cols", [(24, 1500, 64), (300, 1500, 64), (300, 10007, 64), (300, 10007, 72), (1100, 5000, 64)])
def test_entries_far_below_the_label(tokens, vocab, cols, gap):
    """Rows that are sure of their label: what is left for the entries beside it keeps its bits."""
    p = hp.problem(tokens, vocab, cols, gap, device=DEV)
    r = hp.exact(*p)
    for dw_type in (F32, BF16):
        dh, dw = gradients(*p, dw_type)
        assert hp.outside(dw, r["dw"], r["dw_off"]) == 0
        assert hp.outside(dh, r["dh"], r["dh_off"]) == 0


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1000, 64), (24, 2000, 64), (24, 2000, 72), (32, 3001, 200), (40, 2000, 72), (60, 2000, 64),
                                               (200, 4000, 64), (200, 4000, 72), (600, 9001, 64), (600, 20000, 72), (1100, 30011, 128)])
def test_g_at_the_label_has_16_bits(tokens, vocab, cols):
    """Few tokens and more, logits that stay and exponentials that do, weights as they lie and packed."""
    p = hp.problem(tokens, vocab, cols, device=DEV)
    r = hp.exact(*p)
    for dw_type in (F32, BF16):
        dh, dw = gradients(*p, dw_type)
        assert hp.outside(dw, r["dw"], r["dw_off"]) == 0
        assert hp.outside(dh, r["dh"], r["dh_off"]) == 0
    # The bound is one that g without its correction does not keep.
    dh, dw = hp.simulate(*p, correction=0.0)
    assert hp.outside(dw, r["dw"], r["dw_off"]) > 0


@pytest.mark.parametrize("tokens,vocab,cols", [(24, 1500, 64), (24, 1500, 72), (300, 1500, 64), (300, 10007, 64), (300, 10007, 72)])
def test_a_logit_of_minus_infinity(tokens, vocab, cols):
    """It has no part in its row's sum; what it touches of the gradients is NaN, and so is a row with one of plus infinity."""
    hidden, weight, labels, c = hp.problem(tokens, vocab, cols, device=DEV)
    entry = int((labels[0] + 1) % vocab)
    labels[labels == entry] = labels[0].clone()
    weight[entry, 5] = float("inf")
    hidden[:, 5] = -hidden[:, 5].abs() - 0.1
    hidden[3, 5] = 0.5
    ws = torch.empty(mps.linear_cross_entropy_workspace_bytes(tokens, vocab, cols, BF16), dtype=torch.uint8, device=DEV).fill_(255)
    loss, logp, dh, dw = torch.empty(1, device=DEV), torch.empty(tokens, device=DEV), torch.empty_like(hidden), torch.empty(vocab, cols, device=DEV)
    rest = torch.arange(tokens, device=DEV) != 3
    c[3] = 0
    mps.linear_cross_entropy(hidden, weight, labels, c, loss, ws, dhidden=dh, dweight=dw, token_logp=logp)
    without = torch.cat([weight[:entry], weight[entry + 1:]])
    r = hp.exact(hidden[rest], without, torch.where(labels > entry, labels - 1, labels)[rest], c[rest])
    want = torch.log_softmax(hidden[rest].double() @ without.double().t(), 1)
    want = want.gather(1, torch.where(labels > entry, labels - 1, labels)[rest, None])[:, 0]
    off = 2 * (cols + 16) * hp.UNIT * (hidden[rest].double().abs() @ without.double().abs().t()).amax(1) + (128 + 8) * hp.UNIT
    assert hp.outside(logp[rest], want, off) == 0 and torch.isfinite(loss).all()
    others = torch.arange(cols, device=DEV) != 5
    assert hp.outside(dh[rest][:, others], r["dh"][:, others], r["dh_off"][:, others]) == 0 and torch.isnan(dh[rest, 5]).all()
    assert hp.outside(torch.cat([dw[:entry], dw[entry + 1:]]), r["dw"], r["dw_off"]) == 0 and (dw[entry] == 0).all()
    c[3] = 1
    mps.linear_cross_entropy(hidden, weight, labels, c, loss, ws, dhidden=dh, dweight=dw, token_logp=logp)
    assert torch.isnan(logp[3]) and torch.isnan(dh[3]).all() and torch.isnan(loss).all() and hp.outside(logp[rest], want, off) == 0
