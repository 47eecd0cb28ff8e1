"""The operators before the step at the edges of what their header allows: in
place for both types and every kernel, the widest and the tallest matrices,
masked rows among many, and the log-probabilities' own values."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import test_gpu_policy as pol
import train_reference as ref
from test_gpu_act8 import DEV, TYPES, chain, check_frames, framed, gen, near, norm_inputs, randn, rounded
from test_gpu_policy import INF
from train_reference import U

pytestmark = pytest.mark.gpu
WIDEST = 1 << 27
TALL = (1 << 22) + 5


def workspace(n):
    return torch.empty(max(256, n), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------ in place ---

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("alias", ["dy", "residual"])
@pytest.mark.parametrize("rows,cols", [(70, 333), (40, 1000), (600, 2048), (9, 4104), (5, 8200), (7, 16384), (4, 16392), (3, 33001)])
def test_norm_backward_over_its_inputs(dtype, alias, rows, cols):
    g = gen(rows + cols)
    x, w = norm_inputs(g, rows, cols, dtype)
    codes, scales = mps.act8_save(x, *mps.act8_empty(rows, cols, DEV))
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dy, res = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype)
    ws = workspace(mps.act8_rmsnorm_backward_workspace_bytes(rows, cols))
    apart, apart_dw = torch.empty_like(dy), torch.empty(cols, device=DEV)
    mps.act8_rmsnorm_backward(dy, codes, scales, rstd, w, apart, apart_dw, ws, residual_grad=res)
    d, d_whole = framed(rows, cols, dtype)
    r, r_whole = framed(rows, cols, dtype, pad=5)
    d.copy_(dy)
    r.copy_(res)
    dx, dw = (d if alias == "dy" else r), torch.empty(cols, device=DEV)
    mps.act8_rmsnorm_backward(d, codes, scales, rstd, w, dx, dw, ws, residual_grad=r)
    assert torch.equal(dx, apart) and torch.equal(dw, apart_dw)
    assert torch.equal(r, res) if alias == "dy" else torch.equal(d, dy)
    check_frames(d_whole, rows, cols)
    check_frames(r_whole, rows, cols, pad=5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("over", ["dgate", "dup"])
@pytest.mark.parametrize("rows,cols", [(50, 333), (3, 31), (600, 1000)])
def test_swiglu_backward_over_dout(dtype, over, rows, cols):
    g = gen(rows)
    kg, ku = (mps.act8_save(randn(g, rows, cols), *mps.act8_empty(rows, cols, DEV)) for _ in range(2))
    dout = randn(g, rows, cols, dtype=dtype)
    want = mps.act8_swiglu_backward(dout, *kg, *ku, torch.empty_like(dout), torch.empty_like(dout))
    d, d_whole = framed(rows, cols, dtype)
    other, other_whole = framed(rows, cols, dtype, pad=5)
    d.copy_(dout)
    got = mps.act8_swiglu_backward(d, *kg, *ku, *((d, other) if over == "dgate" else (other, d)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_frames(d_whole, rows, cols)
    check_frames(other_whole, rows, cols, pad=5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(700, 1003), (3, 128255), (70, 9001), (70, 20007), (70, 70001)])
def test_the_gradient_over_the_logits_stays_within_them(dtype, rows, vocab):
    whole = torch.full((rows + 2, vocab + 9), 7.0, dtype=dtype, device=DEV)
    s = pol.inputs(gen(rows), rows, vocab, dtype)
    apart = pol.call(s)["dlogits"].clone()
    x = whole[1:1 + rows, 5:5 + vocab]
    x.copy_(s["x"])
    s["x"] = x
    assert torch.equal(pol.call(s, inplace=True)["dlogits"], apart)
    whole[1:1 + rows, 5:5 + vocab] = 7.0
    assert (whole == 7.0).all(), "written outside the logits"


# --------------------------------------------------- the policy loss's rows ---

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [1, 40])
@pytest.mark.parametrize("vocab", [40, 3007, 8192, 12001, 30011, 70001])
def test_masked_rows_among_many(dtype, many, vocab):
    """Twelve kinds of rows, once or forty times over: every row's outputs and the
    loss against 64 bits, and the repeated rows the same bits."""
    s = pol.inputs(gen(vocab), 12, vocab, dtype)
    x, labels = s["x"], s["labels"]
    labels[:] = vocab - 1
    s["weight"][:] = 0.5
    s["adv"] = torch.randn(12, generator=gen(1), device=DEV)
    low = torch.finfo(dtype).min
    x[0, :vocab - 1] = -INF              # one token left
    x[1, :vocab // 2] = -INF
    x[2, :vocab // 2] = low
    x[3] = -INF                          # nothing left: left out
    x[4] = low                           # all alike
    x[5] = float("nan")
    labels[5] = -1                       # left out
    x[6], s["weight"][6] = INF, 0.0      # left out
    x[7, :-1] = low
    x[8] = 0.0
    x[9, ::2] = -INF                     # of an odd vocabulary, the label too
    x[10] += 1000.0
    x[11] -= 1000.0
    logp = torch.log_softmax(x.double(), 1).gather(1, labels.clamp(0)[:, None])[:, 0]
    s["old"] = torch.where(torch.isfinite(logp), logp - 0.05, torch.zeros_like(logp)).float()
    s["ref"] = s["old"] + 0.2
    if many > 1:
        s = {k: v.repeat(many, *[1] * (v.dim() - 1)) for k, v in s.items()}
    want, got = pol.reference(s), pol.call(s)
    assert want["live"].sum() == 9 * many
    live = want["live"]
    if vocab % 2:
        hidden = torch.arange(9, 12 * many, 12, device=DEV)
        assert (got["logp"][hidden] == -INF).all() and (got["kl"][hidden] == INF).all() and got["loss"] == INF
        rest = torch.ones_like(live)
        rest[hidden] = False
        got = {k: v[rest] for k, v in got.items() if k != "loss"}
        s = {k: v[rest] for k, v in s.items()}
        want = pol.reference(s)
        got["loss"] = pol.call(s)["loss"]
        live = want["live"]
    pol.check(s, got, want)
    for k in ("logp", "kl", "dlogits"):
        assert torch.isfinite(got[k].float()).all() and not got[k][~live].any(), k
        parts = got[k].reshape(many, -1)
        assert (parts == parts[0]).all(), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (300, 2051), (5, 8200), (66, 8193), (3, 32769), (70, 20007), (70, 70001), (2, 200003)])
def test_token_logprobs(dtype, rows, vocab):
    """Within the bound of a row's sum, (6 R + 64) u for a range R, and one rounding."""
    s = pol.inputs(gen(vocab), rows, vocab, dtype)
    out = torch.full((rows + 1,), 7.0, device=DEV)
    if rows > 4:
        s["x"][0] = -INF
    mps.token_logprobs(s["x"], s["labels"], out[:rows], workspace(mps.policy_loss_workspace_bytes(rows, vocab)))
    x = s["x"].double()
    left_out = (s["labels"] < 0) | (s["labels"] >= vocab) | (x == -INF).all(1)
    want = (x.gather(1, s["labels"].clamp(0, vocab - 1)[:, None])[:, 0] - torch.logsumexp(x, 1)).masked_fill(left_out, 0.0)
    span = (x.amax(1) - x.amin(1)).nan_to_num(nan=0.0)
    assert ((out[:rows].double() - want).abs() <= (6 * span + 64) * U + want.abs() * U).all()
    assert not out[:rows][left_out].any() and out[rows] == 7


# ------------------------------------------------------ the largest matrices ---

@pytest.mark.parametrize("dtype", TYPES)
def test_widest_rows_kept_and_gated(dtype):
    """One row of 2^27 elements gives the bytes and values of its parts as rows."""
    g = gen(1)
    parts = (1 << 15, 1 << 12)
    a, b = (randn(g, 1, WIDEST, dtype=dtype, scale=3.0) for _ in range(2))
    kept, kept_parts = mps.act8_empty(1, WIDEST, DEV), mps.act8_empty(*parts, DEV)
    mps.act8_save(a, *kept)
    mps.act8_save(a.view(parts), *kept_parts)
    assert torch.equal(kept[0].view(-1), kept_parts[0].view(-1)) and torch.equal(kept[1].view(-1), kept_parts[1].view(-1))
    back, back_parts = torch.empty_like(a), torch.empty(parts, dtype=dtype, device=DEV)
    mps.act8_load(*kept, back)
    mps.act8_load(*kept_parts, back_parts)
    assert torch.equal(back.view(-1), back_parts.view(-1))
    up, up_parts = mps.act8_empty(1, WIDEST, DEV), mps.act8_empty(*parts, DEV)
    mps.act8_swiglu(a, b, back, *kept, *up)
    mps.act8_swiglu(a.view(parts), b.view(parts), back_parts, *kept_parts, *up_parts)
    assert torch.equal(back.view(-1), back_parts.view(-1)) and torch.equal(up[0].view(-1), up_parts[0].view(-1))
    other, other_parts = torch.empty_like(a), torch.empty(parts, dtype=dtype, device=DEV)
    mps.act8_swiglu_backward(a, *kept, *up, back, other)
    mps.act8_swiglu_backward(a.view(parts), *kept_parts, *up_parts, back_parts, other_parts)
    assert torch.equal(back.view(-1), back_parts.view(-1)) and torch.equal(other.view(-1), other_parts.view(-1))


@pytest.mark.parametrize("dtype", TYPES)
def test_widest_norm(dtype):
    g = gen(2)
    x, w = randn(g, 1, WIDEST, dtype=dtype), 1 + 0.1 * torch.randn(WIDEST, generator=g, device=DEV)
    y, rstd, kept = torch.empty_like(x), torch.empty(1, device=DEV), mps.act8_empty(1, WIDEST, DEV)
    mps.act8_rmsnorm(x, w, 1e-5, y, rstd, *kept)
    r = (x.double().square().mean() + 1e-5).rsqrt()
    assert (rstd.double() - r).abs() <= r * ((chain(WIDEST) + 1) / 2 + 5) * U
    want = x.double() * rstd.double() * w.double()
    near(y, want, rounded(want, dtype, 2 * U), "y")
    del y, want
    dy, dx, dw = randn(g, 1, WIDEST, dtype=dtype), torch.empty_like(x), torch.empty(WIDEST, device=DEV)
    mps.act8_rmsnorm_backward(dy, *kept, rstd, w, dx, dw, workspace(mps.act8_rmsnorm_backward_workspace_bytes(1, WIDEST)))
    xh = mps.act8_load(*kept, torch.empty(1, WIDEST, device=DEV)).double() * rstd.double()
    gw = dy.double() * w.double()
    mean = (gw * xh).mean()
    want = rstd.double() * (gw - xh * mean)
    size = rstd.double() * (gw.abs() + xh.abs() * (gw * xh).abs().mean())
    near(dx, want, rounded(want, dtype, 0, size * (chain(WIDEST) + 10) * U), "dx")
    want = (dy.double() * xh)[0]
    near(dw, want, want.abs() * 3 * U, "dweight")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [2, 66])
def test_widest_vocabulary(dtype, rows):
    """2^27 logits, for blocks that share a row and for a row per block: whole numbers of
    equal logits, whose sums are exact whatever their order."""
    if rows > 2 and dtype is torch.float32:
        rows = 65
    x = torch.zeros(rows, WIDEST, dtype=dtype, device=DEV)
    labels = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
    labels[0], labels[rows - 1] = WIDEST - 1, 5
    x[rows - 1, 1 << 26:] = -INF
    one = torch.ones(rows, device=DEV)
    logp = torch.zeros(rows, dtype=torch.float64, device=DEV)
    logp[0] = -torch.log(torch.tensor(float(WIDEST), dtype=torch.float64))
    logp[rows - 1] = -torch.log(torch.tensor(float(1 << 26), dtype=torch.float64))
    loss, lp = torch.empty(1, device=DEV), torch.empty(rows, device=DEV)
    mps.policy_loss(x, labels, logp.float(), one, one, loss, workspace(mps.policy_loss_workspace_bytes(rows, WIDEST)), dlogits=x, token_logp=lp)
    assert ((lp.double() - logp).abs() <= logp.abs() * U * 1.001).all()
    ratio = torch.exp(logp - logp.float().double())
    want = -(ratio[0] + ratio[rows - 1])
    assert (loss[0].double() - want).abs() <= want.abs() * U * 1.001
    half = ref.half_step(dtype)
    for row, there in ((0, WIDEST), (rows - 1, 1 << 26)):
        d = x[row]
        p = ratio[row] / there
        label = int(labels[row])
        assert abs(d[label].double() - (p - ratio[row])) <= ratio[row] * (half + 4 * U)
        d[label] = p.to(dtype)
        assert ((d[:there].double() - p).abs() <= p * (half + 4 * U)).all() and not d[there:].any()
    assert not x[1:rows - 1].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,n,k", [(3, 1, WIDEST), (3, WIDEST, 1), (TALL, 1, 1), (TALL, 9, 33)])
def test_widest_and_longest_weight_gradients(dtype, t, n, k):
    """Whole numbers, below 2^24 in every partial sum: bitwise."""
    g = gen(4)
    small = lambda *shape: torch.randint(-1, 2, shape, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    x, dy = small(t, k), small(t, n).to(dtype)
    codes, scales = mps.act8_save(x.to(torch.bfloat16), *mps.act8_empty(t, k, DEV))
    dw = torch.empty(n, k, device=DEV)
    mps.act8_weight_grad(dy, codes, scales, dw, workspace(mps.act8_weight_grad_workspace_bytes(t, n, k)))
    want = torch.zeros(n, k, device=DEV)
    for i in range(0, t, 1 << 18):
        want += torch.mm(dy[i:i + (1 << 18)].float().t().contiguous(), x[i:i + (1 << 18)].float()) if t > 3 else \
            sum(dy[j].float()[:, None] * x[j].float()[None, :] for j in range(3))
    assert torch.equal(dw, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_tallest_columns(dtype):
    """Millions of rows of one element."""
    g = gen(6)
    x = randn(g, TALL, 1, dtype=dtype)
    kept = mps.act8_empty(TALL, 1, DEV)
    mps.act8_save(x, *kept)
    back = mps.act8_load(*kept, torch.empty(TALL, 1, device=DEV))
    near(back, x.float(), x.double().abs().cpu() * 2.0 ** -4, "read back")
    y, rstd, w = torch.empty_like(x), torch.empty(TALL, device=DEV), torch.full((1,), 0.5, device=DEV)
    mps.act8_rmsnorm(x, w, 1e-5, y, rstd, *kept)
    want, r = ref.rmsnorm(x.double(), w.double(), 1e-5)
    rel = ((chain(1) + 1) / 2 + 5) * U
    near(rstd, r, r.cpu() * rel, "rstd")
    near(y, want, rounded(want, dtype, rel + 2 * U), "y")
    labels = torch.zeros(TALL, dtype=torch.int64, device=DEV)
    labels[::3] = 1
    one, loss = torch.ones(TALL, device=DEV), torch.empty(1, device=DEV)
    lp, d = torch.full((TALL,), 7.0, device=DEV), torch.full_like(x, 7.0)
    mps.policy_loss(x, labels, one * 0, one, one, loss, workspace(mps.policy_loss_workspace_bytes(TALL, 1)), dlogits=d, token_logp=lp)
    # One token: l = 0 and a ratio of 1 in every row that takes part, no gradient in any.
    assert not lp.any() and not d.any()
    taking_part = int((labels == 0).sum())
    assert abs(loss.item() + taking_part) <= taking_part * U
