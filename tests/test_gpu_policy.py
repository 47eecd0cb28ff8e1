"""The policy loss and the labels' log-probabilities on the GPU, against the
64-bit form.

Bounds, u = 2^-24: an exponent (x - max) log2(e) of at most R / ln 2 is off by
3 u of itself, the power by 1 ulp, and joining shares multiplies by powers
whose exponents sum to at most R: each e^(x - max) is within (6 R + 64) u,
R the range of a row's finite logits, and so is their sum.  That is E below:
l is off by E (and one rounding), a ratio or e^d by E relative."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref
from train_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
TYPES = [torch.bfloat16, torch.float32]
SHAPES = [(1, 1), (1, 2), (3, 7), (5, 8), (2, 33), (40, 1000), (7, 2048), (300, 2051), (2, 8192), (5, 8200), (3, 32003), (2, 32768), (3, 32769), (64, 33001), (24, 50257),
          (1, 65536), (4, 65544), (2, 128256), (3, 131072), (2, 131080), (1, 200003), (1100, 515), (2300, 64),
          # more than 64 rows: a row per block, read twice or kept, at both sides of every border and past all that is kept
          (66, 8193), (70, 9001), (65, 16384), (70, 16392), (68, 20007), (65, 32760), (66, 32768), (70, 33001), (300, 40009),
          (65, 65528), (66, 65536), (67, 65545), (70, 128256), (65, 131072), (66, 131080), (65, 140003), (600, 17000)]
LOW, HIGH, KL = 0.2, 0.3, 0.05


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def inputs(g, rows, vocab, dtype, scale=2.0, pad=3):
    """Framed logits and the row vectors; ratios stay off the clip's borders."""
    whole = torch.full((rows + 2, vocab + 2 * pad), float("nan"), dtype=dtype, device=DEV)
    x = whole[1:1 + rows, pad:pad + vocab]
    x.copy_(torch.randn(rows, vocab, generator=g, device=DEV) * scale)
    labels = torch.randint(vocab, (rows,), generator=g, device=DEV)
    logp = (x.double().gather(1, labels[:, None])[:, 0] - torch.logsumexp(x.double(), 1))
    # e^shift: 0.57, 0.74, 0.9, 1.0, 1.1, 1.2, 1.42, 1.73
    shifts = torch.tensor([-0.56, -0.3, -0.1, 0.0, 0.1, 0.18, 0.35, 0.55], device=DEV)
    old = (logp - shifts[torch.randint(8, (rows,), generator=g, device=DEV)]).float()
    s = {"x": x, "labels": labels, "old": old,
         "ref": (logp + 0.4 * torch.randn(rows, generator=g, device=DEV)).float(),
         "adv": torch.randn(rows, generator=g, device=DEV), "weight": torch.rand(rows, generator=g, device=DEV) + 0.1}
    if rows > 4:
        labels[1], labels[2] = -100, vocab
        s["weight"][3] = 0
        s["adv"][4] = 0
    return s


def near_rows(a, b):
    """The same rows by another kernel, whose sums have another order."""
    finite = torch.isfinite(b)
    return torch.equal(finite, torch.isfinite(a)) and bool(((a - b)[finite].abs() <= 1e-5 * (1 + b[finite].abs())).all())


def call(s, grad=True, with_ref=True, workspace=None, inplace=False, **kw):
    x = s["x"]
    rows, vocab = x.shape
    ws = torch.full((max(1, mps.policy_loss_workspace_bytes(rows, vocab)),), 255, dtype=torch.uint8, device=DEV) if workspace is None else workspace
    loss = torch.full((2,), 7.0, device=DEV)
    lp, kl = torch.full((rows + 1,), 7.0, device=DEV), torch.full((rows + 1,), 7.0, device=DEV)
    whole = torch.full((rows + 2, vocab + 10), 7.0, dtype=x.dtype, device=DEV)
    d = x if inplace else whole[1:1 + rows, 5:5 + vocab]
    mps.policy_loss(x, s["labels"], s["old"], s["adv"], s["weight"], loss[:1], ws, clip_low=LOW, clip_high=HIGH,
                    ref_logp=s["ref"] if with_ref else None, kl_coef=KL if with_ref else 0.0, dlogits=d if grad else None,
                    token_logp=lp[:rows], token_kl=kl[:rows], **kw)
    assert loss[1] == 7 and lp[rows] == 7 and kl[rows] == 7
    if grad and not inplace:
        mask = torch.ones_like(whole, dtype=torch.bool)
        mask[1:1 + rows, 5:5 + vocab] = False
        assert (whole[mask] == 7).all(), "written outside dlogits"
    return {"loss": loss[0], "logp": lp[:rows], "kl": kl[:rows], "dlogits": d if grad else None}


def reference(s, with_ref=True):
    return ref.policy(s["x"], s["labels"], s["old"], s["adv"], s["weight"], LOW, HIGH,
                      s["ref"] if with_ref else None, KL if with_ref else 0.0)


def check(s, got, want, with_ref=True):
    x = s["x"].double()
    live = want["live"]
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    span = (finite.amax(1) - torch.where(torch.isfinite(x), x, torch.full_like(x, INF)).amin(1)).clamp(0, 120)
    E = torch.where(live, (6 * span + 64) * U, torch.zeros_like(span))
    logp, kl = want["logp"], want["kl"]
    assert ((got["logp"].double() - logp).abs() <= E + logp.abs() * U).all()
    ratio = torch.exp(logp - s["old"].double())
    q = torch.exp(s["ref"].double() - logp) if with_ref else torch.zeros_like(logp)
    assert ((got["kl"].double() - kl).abs() <= (E * (q + 1) + kl.abs() * U) * 1.01).all()
    w = s["weight"].double() * live
    # What a change of l by E does to a row's loss, and to its slope.
    move = w * E * 1.01 * ((ratio * s["adv"].double()).abs() + KL * (q + 1))
    total = (move + want["row_loss"].abs() * 2.0 ** -40).sum() + want["loss"].abs() * U
    assert (got["loss"].double() - want["loss"]).abs() <= total
    if got["dlogits"] is None:
        return
    d = want["dlogits"]
    hot = torch.zeros_like(d)
    hot[torch.arange(len(live), device=DEV), s["labels"].clamp(0, d.shape[1] - 1)] = 1.0
    # slope * (onehot - p): the slope's own error, p's 2 E, four roundings, one to the type.
    size = (move[:, None] + want["slope"].abs()[:, None] * 4 * U) * (want["p"] + hot) + want["slope"].abs()[:, None] * want["p"] * 2 * E[:, None]
    tiny = torch.finfo(s["x"].dtype).smallest_normal
    bound = size * 1.01 + d.abs() * ref.half_step(s["x"].dtype) + tiny
    off = (got["dlogits"].double() - d).abs() - bound
    assert (off <= 0).all(), f"dlogits {off.max().item():.3e} over its bound"
    assert (got["dlogits"][~live] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_ref", [True, False])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_loss_and_gradient(dtype, rows, vocab, with_ref):
    s = inputs(gen(rows * 31 + vocab), rows, vocab, dtype)
    check(s, call(s, with_ref=with_ref), reference(s, with_ref), with_ref)


@pytest.mark.parametrize("rows,vocab", [(3, 1000), (600, 300), (2, 128256), (2, 140000), (300, 10000), (600, 20000), (300, 128256)])
def test_without_a_gradient_the_values_are_the_same(rows, vocab):
    s = inputs(gen(1), rows, vocab, torch.bfloat16)
    a, b = call(s), call(s, grad=False)
    for k in ("loss", "logp", "kl"):
        assert torch.equal(a[k], b[k]), k
    out = torch.full((rows + 1,), 7.0, device=DEV)
    ws = torch.empty(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV)
    mps.token_logprobs(s["x"], s["labels"], out[:rows], ws)
    want = reference(s)["live"] & (s["weight"] != 0)
    assert torch.equal(out[:rows][want], a["logp"][want]) and out[rows] == 7
    bad = (s["labels"] < 0) | (s["labels"] >= vocab)
    assert (out[:rows][bad] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 77), (700, 1003), (3, 128256), (2, 200003), (300, 9001), (600, 33003), (300, 128256)])
def test_gradient_over_the_logits(dtype, rows, vocab):
    s = inputs(gen(2), rows, vocab, dtype)
    a = call(s)["dlogits"].clone()
    assert torch.equal(call(s, inplace=True)["dlogits"], a)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [1, 40])
@pytest.mark.parametrize("vocab", [40, 3000 + 7, 12001, 30011, 70001, 131072])
def test_masked_logits_and_rows(dtype, vocab, many):
    """-inf and lowest-value masks, rows of them alone, and values in rows that are
    left out; in a few rows, and in enough for the kernels of many rows."""
    s = inputs(gen(vocab), 12, vocab, dtype)
    x, labels = s["x"], s["labels"]
    labels[:] = vocab - 1
    s["weight"][:] = 0.5
    s["adv"][:] = torch.randn(12, device=DEV)
    low = torch.finfo(dtype).min
    x[0, :vocab - 1] = -INF              # one token left: p = 1
    x[1, :vocab // 2] = -INF
    x[2, :vocab // 2] = low
    x[3] = -INF                          # nothing left: left out
    x[4] = low                           # all alike: uniform
    x[5] = float("nan")
    labels[5] = -1                       # left out, its logits are not read
    x[6], s["weight"][6] = INF, 0.0
    x[7, :-1] = low
    x[8] = 0.0
    x[9, ::2] = -INF
    x[10] += 1000.0
    x[11] -= 1000.0
    logp = torch.log_softmax(x.double(), 1)[:, -1]
    s["old"] = torch.where(torch.isfinite(logp), logp - 0.05, torch.zeros_like(logp)).float()
    s["ref"] = s["old"] + 0.2
    want = reference(s)
    assert not want["live"][[3, 5, 6]].any() and want["live"].sum() == 9
    if many > 1:
        once = call(s)
        several = call({k: v.repeat(many, *[1] * (v.dim() - 1)) for k, v in s.items()})
        for i in range(many):
            for k in ("logp", "kl"):
                a, b = several[k][i * 12:i * 12 + 12], once[k]
                assert torch.equal(torch.nan_to_num(a, nan=1e9, posinf=1e30, neginf=-1e30),
                                   torch.nan_to_num(b, nan=1e9, posinf=1e30, neginf=-1e30)) or near_rows(a, b), (i, k)
        got = {k: v[12 * (many - 1):] for k, v in several.items() if k != "loss"}
        got["loss"] = once["loss"]
    else:
        got = call(s)
    if vocab % 2:
        # Row 9's label is masked itself: an infinite KL term in its own outputs and the loss.
        assert got["logp"][9] == -INF and got["kl"][9] == INF and got["loss"] == INF
        assert not torch.isfinite(want["loss"])
        keep = [i for i in range(12) if i != 9]
        s = {k: v[keep] for k, v in s.items()}
        want = reference(s)
        got = {k: v[keep] for k, v in got.items() if k != "loss"}
        got["loss"] = call(s)["loss"]
    assert torch.isfinite(got["dlogits"].float()).all()
    check(s, got, want)
    for i in (3, 5, 6):
        assert got["logp"][i] == 0 and got["kl"][i] == 0
    assert got["logp"][0] == 0 and got["logp"][7] == 0


@pytest.mark.parametrize("rows,vocab", [(600, 100), (3, 128256), (70, 12000), (70, 20000), (70, 128256)])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_nonfinite_logits_make_their_row_nan(rows, vocab, bad):
    s = inputs(gen(4), rows, vocab, torch.float32 if vocab == 100 else torch.bfloat16)
    s["labels"][:] = 5
    s["weight"][:], s["adv"][:] = 1.0, 1.0
    s["x"][2, vocab // 2] = bad
    got = call(s)
    assert torch.isnan(got["logp"][2]) and torch.isnan(got["dlogits"][2].float()).all() and torch.isnan(got["loss"])
    others = [i for i in range(s["x"].shape[0]) if i != 2]
    assert torch.isfinite(got["logp"][others]).all() and torch.isfinite(got["dlogits"][others].float()).all()


def test_a_label_that_is_masked():
    """l = -inf: no ratio, and an infinite KL term where there is one."""
    s = inputs(gen(6), 1, 50, torch.float32)
    s["x"][0, 9] = -INF
    s["labels"][:], s["adv"][:], s["old"][:] = 9, 1.0, -3.0
    got = call(s, with_ref=False)
    assert got["logp"][0] == -INF and got["loss"] == 0 and not got["dlogits"].any()


def test_extreme_ratios():
    s = inputs(gen(8), 6, 64, torch.float32)
    s["labels"][:], s["weight"][:] = 3, 1.0
    s["adv"] = torch.tensor([1.0, -1.0, 0.0, 1.0, -1.0, 0.0], device=DEV)
    s["old"] = torch.tensor([-2000.0, -2000.0, -2000.0, 2000.0, 2000.0, 2000.0], device=DEV)
    got = call(s, with_ref=False)
    d = got["dlogits"]
    assert (d[[0, 2, 3, 4, 5]] == 0).all()  # clipped, no advantage, or a ratio of 0
    assert not torch.isfinite(d[1]).all() and got["loss"] == INF
    s["adv"][1] = 0.0
    # rows 0 and 4 pay (1 + high) and (1 - low), rows 2, 5 and 1 nothing, row 3 ratio 0
    assert abs(call(s, with_ref=False)["loss"].item() - (-(1 + HIGH) + (1 - LOW))) <= 2 * U * 2


@pytest.mark.parametrize("rows", [0, 1, 2000])
@pytest.mark.parametrize("vocab", [300, 9000, 20000])
def test_rows_that_are_all_left_out(rows, vocab):
    s = inputs(gen(1), max(rows, 1), vocab, torch.bfloat16)
    s = {k: (v[:rows] if k != "x" else v[:rows]) for k, v in s.items()}
    s["labels"] = torch.full_like(s["labels"], -100)
    s["x"][:] = float("nan")
    got = call(s)
    assert got["loss"] == 0 and not got["logp"].any() and not got["kl"].any() and not got["dlogits"].any()


@pytest.mark.parametrize("rows,vocab", [(6, 128256), (3000, 900), (700, 10000), (700, 30000), (300, 128256)])
def test_two_runs_give_the_same_bits(rows, vocab):
    s = inputs(gen(7), rows, vocab, torch.bfloat16)
    a = call(s)
    b = call(s, workspace=torch.zeros(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV))
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("vocab", [131072, 1000])
def test_more_than_2_to_the_32_logits(vocab):
    rows = (1 << 32) // vocab + 3
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device=DEV)
    s = inputs(gen(9), 3, vocab, torch.bfloat16)
    x[-3:] = s["x"]
    labels = torch.full((rows,), -1, device=DEV)
    labels[-3:] = s["labels"]
    one = {"x": x, "labels": labels}
    for k in ("old", "ref", "adv", "weight"):
        one[k] = torch.zeros(rows, device=DEV)
        one[k][-3:] = s[k]
    want = reference(s)
    ws = torch.empty(mps.policy_loss_workspace_bytes(rows, vocab), dtype=torch.uint8, device=DEV)
    loss, lp = torch.empty(1, device=DEV), torch.empty(rows, device=DEV)
    mps.policy_loss(x, labels, one["old"], one["adv"], one["weight"], loss, ws, clip_low=LOW, clip_high=HIGH,
                    ref_logp=one["ref"], kl_coef=KL, dlogits=x, token_logp=lp)
    got = {"loss": loss[0], "logp": lp[-3:], "kl": want["kl"].float(), "dlogits": x[-3:]}
    check(s, got, want)
    assert not lp[:-3].any() and not x[:-3].any()


def test_refusals():
    s = inputs(gen(1), 4, 64, torch.float32)
    ws = torch.empty(mps.policy_loss_workspace_bytes(4, 64), dtype=torch.uint8, device=DEV)
    loss = torch.zeros(1, device=DEV)
    args = lambda **kw: mps.policy_loss(s["x"], s["labels"], s["old"], s["adv"], s["weight"], loss, **{"workspace": ws, **kw})  # noqa: E731
    with pytest.raises(mps.MpsError, match="clip_low"):
        args(clip_low=1.0)
    with pytest.raises(mps.MpsError, match="kl_coef"):
        args(kl_coef=0.1)
    with pytest.raises(mps.MpsError, match="workspace"):
        args(workspace=None)
    with pytest.raises(mps.MpsError, match="overlap"):
        args(token_logp=s["old"])
    with pytest.raises(ValueError, match="dlogits"):
        args(dlogits=torch.empty(4, 63, device=DEV))
    with pytest.raises(TypeError, match="dlogits"):
        args(dlogits=torch.empty(4, 64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="labels"):
        mps.token_logprobs(s["x"], s["labels"].int(), loss, ws)
    with pytest.raises(mps.MpsError, match="stride"):
        mps.token_logprobs(s["x"][:1].expand(4, 64), s["labels"], torch.empty(4, device=DEV), ws)
