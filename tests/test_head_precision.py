"""The bounds of head_precision on the CPU: the operator's arithmetic in 64 bits
keeps them, and each planted mistake breaks them."""
import pytest
import torch

import head_precision as hp


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1000, 64), (24, 2000, 64), (60, 2000, 72), (200, 4000, 64), (600, 9001, 64)])
def test_the_label_s_correction_shows(tokens, vocab, cols):
    p = hp.problem(tokens, vocab, cols)
    r = hp.exact(*p)
    for kept in (None, "log"):
        dh, dw = hp.simulate(*p, kept=kept)
        assert hp.outside(dh, r["dh"], r["dh_off"]) == 0 and hp.outside(dw, r["dw"], r["dw_off"]) == 0
    for wrong in (0.0, -1.0):
        dh, dw = hp.simulate(*p, correction=wrong)
        assert hp.outside(dw, r["dw"], r["dw_off"]) > 0
        if tokens > 1:
            assert hp.outside(dh, r["dh"], r["dh_off"]) > 0


@pytest.mark.parametrize("gap", [12.0, 18.0, 24.0, 34.0])
def test_exponentials_far_below_the_label_s(gap):
    p = hp.problem(300, 1500, 64, gap)
    r = hp.exact(*p)
    dh, dw = hp.simulate(*p)
    assert hp.outside(dh, r["dh"], r["dh_off"]) == 0 and hp.outside(dw, r["dw"], r["dw_off"]) == 0
    _, dw = hp.simulate(*p, kept="fp16")
    bad = hp.outside(dw, r["dw"], r["dw_off"])
    assert bad == 0 if gap < 14 else bad > 1000
    assert int((p[2] != p[2][0]).sum()) == 0 and torch.isfinite(dw).all()
