"""8-bit activations on the GPU: keeping and reading back bitwise against the
oracle, RMSNorm and SwiGLU forward and backward against the 64-bit forms.

Bounds, with u = 2^-24 (fp32) and h half a step of the output's type:
a value that takes n fp32 roundings is off by at most n u relative; a sum of
n products by (longest chain of additions + 1) u of the sum of magnitudes."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref
from train_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float32]
# One element; a run's borders; odd rows; a wavefront's, a block's and many blocks' worth; long rows.
SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (64, 200), (7, 1001), (300, 515), (33, 2048), (9, 2056), (5, 4104), (4, 8200),
          (3, 16392), (2, 33000), (1, 70001)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def framed(rows, cols, dtype, fill=7.0, pad=3):
    """A matrix inside a larger one (an odd start and stride), and the larger one."""
    whole = torch.full((rows + 2, cols + 2 * pad), fill, dtype=dtype, device=DEV)
    return whole[1:1 + rows, pad:pad + cols], whole


def frame_kept(rows, cols):
    """Codes and scales followed by sentinel bytes."""
    row = mps.act8_row(cols)
    c = torch.full((rows * row + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((rows * row // 32 + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    return c[:rows * row].view(rows, row), s[:rows * row // 32].view(rows, row // 32), c, s


def check_frames(whole, rows, cols, pad=3, fill=7.0):
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[1:1 + rows, pad:pad + cols] = False
    assert (whole[mask] == fill).all(), "written outside the matrix"


def check_kept(codes, scales, want, c=None, s=None):
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    for whole, part in ((c, codes), (s, scales)):
        if whole is not None:
            assert (whole[part.numel():] == 0xA5).all(), "written behind the kept bytes"


def near(got, want, bound, what):
    got, want = got.double().cpu(), want.double().cpu()
    bound = bound.cpu() if torch.is_tensor(bound) else bound
    off = (got - want).abs() - bound
    assert not torch.isnan(got).any(), what
    assert (off <= 0).all(), f"{what}: {off.max().item():.3e} over its bound at {int(off.argmax())}"


def rounded(want, dtype, relative, floor=0.0):
    """|want| (relative + half a step) + floor, with the type's smallest steps."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return want.double().abs() * (relative + ref.half_step(dtype) * (1 + relative)) + floor + tiny


def wide_range(g, rows, cols, dtype):
    """Rows whose runs have magnitudes from 2^-126 to 2^100, zeros among them."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    e = torch.randint(-120, 100, (rows, (cols + 31) // 32), generator=g, device=DEV).repeat_interleave(32, 1)[:, :cols]
    x = torch.ldexp(x, e)
    x[torch.rand(rows, cols, generator=g, device=DEV) < 0.05] = 0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_keep_and_read_back(oracle_lib, dtype, rows, cols):
    g = gen(rows * 100003 + cols)
    x, _ = framed(rows, cols, dtype)
    x.copy_(wide_range(g, rows, cols, dtype))
    codes, scales, c, s = frame_kept(rows, cols)
    mps.act8_save(x, codes, scales)
    check_kept(codes, scales, ref.keep(oracle_lib, x), c, s)
    want = ref.values(codes, scales, cols)
    for out_type in TYPES:
        out, whole = framed(rows, cols, out_type)
        mps.act8_load(codes, scales, out)
        assert torch.equal(out, want.to(torch.float32).to(out_type))
        check_frames(whole, rows, cols)


@pytest.mark.parametrize("dtype", TYPES)
def test_nonfinite_runs(oracle_lib, dtype):
    x = torch.randn(6, 130, device=DEV).to(dtype)
    x[0, 5], x[1, 40], x[2, 129], x[3, 0], x[3, 127] = float("nan"), float("inf"), -float("inf"), float("inf"), float("nan")
    x[4] = torch.finfo(dtype).max
    x[5] = torch.finfo(dtype).smallest_normal
    codes, scales = mps.act8_empty(6, 130, DEV)
    mps.act8_save(x, codes, scales)
    check_kept(codes, scales, ref.keep(oracle_lib, x))
    back = mps.act8_load(codes, scales, torch.empty(6, 130, dtype=torch.float32, device=DEV))
    want = ref.values(codes, scales, 130).float().cpu()
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(back.cpu(), nan=1.0), torch.nan_to_num(want, nan=1.0))
    assert torch.isnan(back[0, :32]).all() and not torch.isnan(back[0, 32:]).any()


def test_every_code_at_every_scale():
    """All 256 codes at all 256 scale bytes, read back as fp32 and bf16."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    want = ref.values(codes, scales, 256)
    f32 = want.float()  # one rounding; 2^-136 .. inf
    for dtype in TYPES:
        out = mps.act8_load(codes.to(DEV), scales.to(DEV), torch.empty(256, 256, dtype=dtype, device=DEV)).cpu()
        w = f32.to(dtype)
        assert torch.equal(torch.isnan(out), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(out, nan=0.0, posinf=1e38, neginf=-1e38),
                           torch.nan_to_num(w, nan=0.0, posinf=1e38, neginf=-1e38))


def chain(cols):
    """Additions a value passes in a row's sum: at most a thread's own (256 threads
    of eight elements), the wavefront's six and sixteen wavefronts'."""
    return 8 * -(-cols // 2048) + 6 + 16


def norm_inputs(g, rows, cols, dtype):
    x = randn(g, rows, cols, dtype=dtype, scale=3.0)
    x[0] *= 1e-6
    w = 1 + 0.3 * torch.randn(cols, generator=g, device=DEV)
    return x, w


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rmsnorm(oracle_lib, dtype, rows, cols):
    g = gen(rows * 7 + cols)
    src, w = norm_inputs(g, rows, cols, dtype)
    x, _ = framed(rows, cols, dtype)
    x.copy_(src)
    y, whole = framed(rows, cols, dtype, pad=5)
    rstd = torch.full((rows + 1,), 7.0, device=DEV)
    codes, scales, c, s = frame_kept(rows, cols)
    mps.act8_rmsnorm(x, w, 1e-5, y, rstd[:rows], codes, scales)
    check_frames(whole, rows, cols, pad=5)
    check_kept(codes, scales, ref.keep(oracle_lib, x), c, s)
    want, r = ref.rmsnorm(x.double(), w.double(), 1e-5)
    # The sum of squares: chain + 1; the mean's division, + eps (and eps itself rounded to fp32), root, reciprocal: 5, the sum's half.
    rel = ((chain(cols) + 1) / 2 + 5) * U
    near(rstd[:rows], r, r.cpu() * rel, "rstd")
    assert rstd[rows] == 7.0
    near(y, want, rounded(want, dtype, rel + 2 * U), "y")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 96), (2100, 40), (0, 64)])
@pytest.mark.parametrize("full", [False, True])
def test_rmsnorm_backward(oracle_lib, dtype, rows, cols, full):
    g = gen(rows * 13 + cols + full)
    x, w = norm_inputs(g, max(rows, 1), cols, dtype)
    x = x[:rows]
    codes, scales = (t.to(DEV) for t in ref.keep(oracle_lib, x))
    codes[:, cols:] = 0x55  # the padding's bytes mean nothing
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dy, _ = framed(rows, cols, dtype)
    dy.copy_(randn(g, rows, cols, dtype=dtype))
    dx, whole = framed(rows, cols, dtype, pad=1)
    dweight = torch.full((cols + 1,), 7.0, device=DEV)
    before = torch.randn(cols, generator=g, device=DEV)
    kw, res, out = {}, None, None
    if full:
        res = randn(g, rows, cols, dtype=dtype)
        out = frame_kept(rows, cols)
        dweight[:cols] = before
        kw = dict(residual_grad=res, accumulate=True, out_codes=out[0], out_scales=out[1])
    ws = torch.empty(max(1, mps.act8_rmsnorm_backward_workspace_bytes(rows, cols)), dtype=torch.uint8, device=DEV)
    mps.act8_rmsnorm_backward(dy, codes, scales, rstd, w, dx, dweight[:cols], ws, **kw)
    check_frames(whole, rows, cols, pad=1)
    assert dweight[cols] == 7.0
    xk = ref.values(codes, scales, cols).to(DEV)
    wd, d, r = w.double(), dy.double(), rstd.double()
    want_dx, want_dw, y = ref.rmsnorm_backward(d, xk, r, wd, res.double() if full else None)
    if rows:
        xh, gw = xk * r[:, None], d * wd
        # g, xh: one rounding each; their product's mean: chain + 4; then two products, a difference, a product, the residual's sum.
        mean = (gw * xh).abs().mean(1, keepdim=True)
        size = r[:, None] * (gw.abs() + xh.abs() * mean) + (res.double().abs() if full else 0)
        near(dx, want_dx, rounded(want_dx, dtype, 0, size * (chain(cols) + 10) * U), "dx")
    # At most all rows in one chain of fp32 additions (and the joining sums of partial rows).
    size = (d * xk * r[:, None]).abs().sum(0) if rows else torch.zeros(cols, device=DEV)
    if full:
        want_dw, size = want_dw + before.double(), size + before.double().abs()
    near(dweight[:cols], want_dw, size * (rows + 1030) * U + 1e-45, "dweight")
    if full and rows:
        # The same two fp32 products as the bytes are made from: bitwise.
        again = xk.float() * rstd[:, None] * w
        check_kept(out[0], out[1], ref.keep(oracle_lib, again), out[2], out[3])


@pytest.mark.parametrize("alias", ["dy", "residual"])
def test_rmsnorm_backward_in_place(oracle_lib, alias):
    g = gen(5)
    rows, cols = 70, 1000
    x, w = norm_inputs(g, rows, cols, torch.bfloat16)
    codes, scales = (t.to(DEV) for t in ref.keep(oracle_lib, x))
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dy, res = randn(g, rows, cols, dtype=torch.bfloat16), randn(g, rows, cols, dtype=torch.bfloat16)
    ws = torch.empty(mps.act8_rmsnorm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    outs = []
    for inplace in (False, True):
        d, r = dy.clone(), res.clone()
        dx = torch.empty_like(dy) if not inplace else (d if alias == "dy" else r)
        dw = torch.empty(cols, device=DEV)
        mps.act8_rmsnorm_backward(d, codes, scales, rstd, w, dx, dw, ws, residual_grad=r)
        outs.append((dx, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_a_nan_in_one_row_stays_there(oracle_lib):
    """A row with a NaN gives NaN in its own outputs only (and in dweight)."""
    x = torch.randn(4, 64, device=DEV)
    x[2, 3] = float("nan")
    codes, scales = mps.act8_empty(4, 64, DEV)
    y, rstd, w = torch.empty_like(x), torch.empty(4, device=DEV), torch.ones(64, device=DEV)
    mps.act8_rmsnorm(x, w, 1e-5, y, rstd, codes, scales)
    assert torch.isnan(y[2]).all() and not torch.isnan(y[[0, 1, 3]]).any()
    ws = torch.empty(mps.act8_rmsnorm_backward_workspace_bytes(4, 64), dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(64, device=DEV)
    mps.act8_rmsnorm_backward(torch.ones_like(x), codes, scales, rstd, w, dx, dw, ws)
    assert torch.isnan(dx[2]).all() and not torch.isnan(dx[[0, 1, 3]]).any() and torch.isnan(dw).all()


def gate_values(g, rows, cols, dtype):
    x = randn(g, rows, cols, dtype=dtype, scale=3.0)
    if cols > 8:
        x[0, :8] = torch.tensor([0.0, -0.0, 90.0, -90.0, 30.0, -30.0, 200.0, -200.0], device=DEV).to(dtype)
    return x


# sigmoid: the exponent's correction leaves 2 u, the power 1 ulp (2 u), 1 + t one u, the reciprocal 1 ulp.
SIG = 8 * U


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_swiglu(oracle_lib, dtype, rows, cols):
    g = gen(rows * 17 + cols)
    both = torch.empty(rows, 2 * cols + 1, dtype=dtype, device=DEV)  # an odd stride
    gate, up = both[:, :cols], both[:, cols:2 * cols]
    gate.copy_(gate_values(g, rows, cols, dtype))
    up.copy_(randn(g, rows, cols, dtype=dtype))
    out, whole = framed(rows, cols, dtype)
    kg, ku = frame_kept(rows, cols), frame_kept(rows, cols)
    mps.act8_swiglu(gate, up, out, kg[0], kg[1], ku[0], ku[1])
    check_frames(whole, rows, cols)
    check_kept(kg[0], kg[1], ref.keep(oracle_lib, gate), kg[2], kg[3])
    check_kept(ku[0], ku[1], ref.keep(oracle_lib, up), ku[2], ku[3])
    want = ref.swiglu(gate.double(), up.double())
    # e^-g overflows fp32 from g = -88.7 down, where the value is below 1e-35.
    near(out, want, rounded(want, dtype, SIG + 2 * U, 1e-35), "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("again", [False, True])
def test_swiglu_backward(oracle_lib, dtype, rows, cols, again):
    g = gen(rows * 19 + cols)
    kg = [t.to(DEV) for t in ref.keep(oracle_lib, gate_values(g, rows, cols, dtype))]
    ku = [t.to(DEV) for t in ref.keep(oracle_lib, randn(g, rows, cols, dtype=dtype))]
    kg[0][:, cols:] = 0x55
    ku[0][:, cols:] = 0x7f  # NaN codes behind the row's end mean nothing
    dout, _ = framed(rows, cols, dtype)
    dout.copy_(randn(g, rows, cols, dtype=dtype))
    both = torch.full((rows, 2 * cols + 1), 7.0, dtype=dtype, device=DEV)
    dgate, dup = both[:, :cols], both[:, cols:2 * cols]
    out = frame_kept(rows, cols)
    kw = dict(out_codes=out[0], out_scales=out[1]) if again else {}
    mps.act8_swiglu_backward(dout, *kg, *ku, dgate, dup, **kw)
    assert (both[:, 2 * cols] == 7.0).all()
    gd, ud, d = ref.values(*kg, cols).to(DEV), ref.values(*ku, cols).to(DEV), dout.double()
    s = 1 / (1 + torch.exp(-gd))
    want_dg, want_du = ref.swiglu_backward(d, gd, ud)
    f = (1 + gd * (1 - s)).abs()
    size = (d * ud * s).abs() * ((SIG + 4 * U) * f + gd.abs() * (SIG * s + 2 * U * (1 - s)) + 2 * U)
    near(dgate, want_dg, rounded(want_dg, dtype, 0, size + 1e-35), "dgate")
    near(dup, want_du, rounded(want_du, dtype, SIG + 2 * U, 1e-35), "dup")
    if again:
        want = ref.swiglu(gd, ud)
        _, sc = ref.keep(oracle_lib, want.float())
        got = ref.values(out[0], out[1], cols).to(DEV)
        # Half a step of E4M3 (2^-4 of a value, 2^-17 of its run's largest), and a value next to the border of a
        # scale may take the next one: then half a step of that.
        run = torch.nn.functional.pad(want, (0, mps.act8_row(cols) - cols)).view(rows, -1, 32).abs().amax(2)
        run = run.repeat_interleave(32, 1)[:, :cols]
        near(got, want, want.abs() * (2.0 ** -4 + SIG * 2) + run * 2.0 ** -16 + 1e-35, "the output again")
        assert (out[1].cpu().int() - sc.int()).abs().max() <= 1
        assert ((out[1].cpu() != sc).float().mean()) < 0.01 + 1.5 / sc.numel()
        assert not out[0][:, cols:].any()
        assert (out[2][out[0].numel():] == 0xA5).all() and (out[3][out[1].numel():] == 0xA5).all()


def test_swiglu_backward_over_dout(oracle_lib):
    g = gen(11)
    kg = [t.to(DEV) for t in ref.keep(oracle_lib, randn(g, 50, 333))]
    ku = [t.to(DEV) for t in ref.keep(oracle_lib, randn(g, 50, 333))]
    dout = randn(g, 50, 333)
    a, b = torch.empty_like(dout), torch.empty_like(dout)
    mps.act8_swiglu_backward(dout, *kg, *ku, a, b)
    for first in (True, False):
        d, other = dout.clone(), torch.empty_like(dout)
        mps.act8_swiglu_backward(d, *kg, *ku, *((d, other) if first else (other, d)))
        assert torch.equal(d if first else other, a) and torch.equal(other if first else d, b)


def test_overlaps_and_strides_are_refused():
    x = torch.zeros(4, 64, device=DEV)
    codes, scales = mps.act8_empty(4, 64, DEV)
    with pytest.raises(mps.MpsError, match="overlap"):
        mps.act8_swiglu(x, x, x, codes, scales, *mps.act8_empty(4, 64, DEV))
    with pytest.raises(mps.MpsError, match="stride"):
        mps.act8_save(x[:1].expand(4, 64), codes, scales)
    with pytest.raises(ValueError, match="contiguous"):
        mps.act8_save(torch.zeros(64, 4, device=DEV).t(), codes, scales)
    with pytest.raises(ValueError, match="scales"):
        mps.act8_save(x, codes, scales[:, :1])
    with pytest.raises(TypeError):
        mps.act8_save(x.half(), codes, scales)


def test_more_than_2_to_the_32_elements():
    """Rows behind the 2^32nd element of codes and matrix are read and written."""
    rows, cols = (1 << 20) + 3, 4128
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(5, cols, device=DEV).to(torch.bfloat16)
    x[-5:] = tail
    codes, scales = mps.act8_empty(rows, cols, DEV)
    codes[-5:], scales[-5:] = 0xA5, 0xA5
    mps.act8_save(x, codes, scales)
    c, s = mps.act8_empty(5, cols, DEV)
    mps.act8_save(tail, c, s)
    assert torch.equal(codes[-5:], c) and torch.equal(scales[-5:], s)
    x.fill_(1)
    mps.act8_load(codes, scales, x)
    assert torch.equal(x[-5:], mps.act8_load(c, s, torch.empty_like(tail)))
    assert not x[:rows - 5].any()
