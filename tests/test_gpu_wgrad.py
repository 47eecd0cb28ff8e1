"""The weight gradient from 8-bit activations on the GPU, against 64 bits.

With small whole numbers every product and sum is exact in fp32 whatever the
order, so those cases are compared bitwise.  Otherwise a sum of n products is
off by at most (n + 8) 2^-23 of the sum of magnitudes (a chain of n fp32
additions that may cut off instead of rounding), plus half a step of dw."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float32]
# (tokens, out, in): one of each; borders of the matrix instruction's 16 x 32 x 32, of tiles of 128 and 256,
# of stages of 32 and 64 tokens; more tokens than one block takes; none.
SHAPES = [(1, 1, 1), (5, 3, 7), (31, 33, 32), (32, 128, 128), (33, 129, 131), (64, 64, 256), (65, 256, 96), (0, 40, 50),
          (100, 8, 2051), (257, 513, 40), (515, 1000, 33), (1030, 260, 520), (2500, 72, 136), (4099, 16, 24), (300, 512, 768),
          (700, 768, 512),
          (257, 1032, 1025), (1030, 520, 2051), (1500, 264, 4000), (12000, 260, 300),
          # tiles of 128, without and with splits of the tokens
          (2048, 2048, 2048), (3000, 1025, 2050),
          # bf16 gradients: tiles of 256, with splits and without, rows of whole 16-byte chunks and odd ones
          (4000, 1032, 2056), (4000, 1031, 2056), (600, 4096, 4352), (700, 4099, 4100),
          # the same for fp32 gradients
          (1, 4096, 4096), (33, 4096, 4100), (450, 2300, 4099), (1000, 2051, 4099), (2047, 2050, 2056), (6000, 1028, 1030),
          (6000, 1031, 1030)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def kept(oracle_lib, x):
    """x in 8 bits: by the oracle, or, where that would take seconds, by act8_save
    (which is compared with the oracle bitwise in its own tests)."""
    if x.numel() < 300000:
        return tuple(v.to(DEV) for v in ref.keep(oracle_lib, x))
    return mps.act8_save(x.to(DEV), *mps.act8_empty(*x.shape, DEV))


def workspace(t, n, k):
    return torch.empty(max(1, mps.act8_weight_grad_workspace_bytes(t, n, k)), dtype=torch.uint8, device=DEV)


def product(dy, codes, scales, k):
    """dy^T x and the sums of magnitudes, in 64 bits."""
    x = ref.values(codes, scales, k).to(DEV)
    d = dy.double()
    return torch.mm(d.t().contiguous(), x.contiguous()), torch.mm(d.abs().t().contiguous(), x.abs().contiguous())


def guarded(n, k, dtype, offset=1):
    """dw at an odd element of a larger buffer, and the buffer."""
    buf = torch.full((n * k + 2 * offset + 8,), 7.0, dtype=dtype, device=DEV)
    return buf[offset:offset + n * k].view(n, k), buf


def check_guard(buf, n, k, offset=1):
    assert (buf[:offset] == 7).all() and (buf[offset + n * k:] == 7).all(), "written outside dw"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dw_type", TYPES)
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_whole_numbers_bitwise(oracle_lib, dtype, dw_type, t, n, k):
    g = gen(t + 3 * n + 7 * k)
    x = torch.randint(-4, 5, (t, k), generator=g, device=DEV).float()
    codes, scales = kept(oracle_lib, x)
    codes[:, k:] = 0x38
    # A matrix inside a larger one: 16-byte rows where n allows them, else an odd start and stride.
    left = 8 if n % 8 == 0 else 3
    wide = torch.randint(-8, 9, (t + 2, n + left + 8), generator=g, device=DEV).to(dtype)
    wide[t:] = float("nan")  # rows behind the last token
    wide[:, n + left:], wide[:, :left] = float("nan"), float("inf")  # columns beside the matrix
    dy = wide[:t, left:n + left]
    want, _ = product(dy, codes, scales, k)
    dw, buf = guarded(n, k, dw_type)
    ws = workspace(t, n, k)
    mps.act8_weight_grad(dy, codes, scales, dw, ws)
    assert torch.equal(dw, want.to(dw_type))
    check_guard(buf, n, k)
    before = torch.randint(-50, 50, (n, k), generator=g, device=DEV).to(dw_type)
    dw.copy_(before)
    mps.act8_weight_grad(dy, codes, scales, dw, ws, accumulate=True)
    assert torch.equal(dw, (want + before.double()).to(dw_type))
    check_guard(buf, n, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,n,k", SHAPES + [(3000, 384, 640), (8200, 130, 70)])
def test_values(oracle_lib, dtype, t, n, k):
    g = gen(5 * t + n + k)
    codes, scales = kept(oracle_lib, torch.randn(t, k, generator=g, device=DEV))
    dy = (torch.randn(t, n, generator=g, device=DEV) * 0.01).to(dtype)
    want, size = product(dy, codes, scales, k)
    dw = torch.empty(n, k, device=DEV)
    mps.act8_weight_grad(dy, codes, scales, dw, workspace(t, n, k))
    assert ((dw.double() - want).abs() <= size * (t + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -24).all()
    # In the mean far nearer than the worst case: an fp32 product, not a bf16 one.
    if t > 16:
        assert (dw.double() - want).norm() <= 4e-6 * want.norm()


def test_fp32_gradients_keep_all_their_bits(oracle_lib):
    """One token and x = 1: dw is dy itself, every bit of it."""
    dy = torch.randn(1, 400, device=DEV)
    dy[0, :6] = torch.tensor([3.4028234e38, -3.4028234e38, 1.1754944e-38, 1.0000001, -0.99999994, 0.0])
    codes, scales = kept(oracle_lib, torch.ones(1, 32))
    dw = torch.empty(400, 32, device=DEV)
    mps.act8_weight_grad(dy, codes, scales, dw, workspace(1, 400, 32))
    assert torch.equal(dw, dy.t().expand(400, 32))


@pytest.mark.parametrize("dtype,t,n,k", [(torch.bfloat16, 70, 150, 160), (torch.float32, 70, 150, 160),
                                         (torch.bfloat16, 600, 4096, 4352), (torch.bfloat16, 700, 4099, 4100),
                                         (torch.float32, 450, 2300, 4099), (torch.float32, 1000, 2051, 4099)])
def test_nonfinite_values_stay_in_their_rows_and_columns(oracle_lib, dtype, t, n, k):
    x = torch.ones(t, k)
    x[3, 40] = float("nan")  # the run of columns 32 .. 63
    dy = torch.ones(t, n, device=DEV, dtype=dtype)
    dy[5, 7], dy[6, 8], dy[9, 9] = float("inf"), -float("inf"), float("nan")
    codes, scales = kept(oracle_lib, x)
    dw = mps.act8_weight_grad(dy, codes, scales, torch.empty(n, k, device=DEV), workspace(t, n, k))
    clean_rows = [i for i in range(n) if i not in (7, 8, 9)]
    clean = torch.ones(k, dtype=torch.bool)
    clean[32:64] = False
    assert torch.isnan(dw[:, 32:64]).all() and torch.isnan(dw[9]).all()
    assert (dw[7][clean] == float("inf")).all() and (dw[8][clean] == -float("inf")).all()
    assert (dw[clean_rows][:, clean] == t).all()


def test_small_and_large_kept_values(oracle_lib):
    """Kept values down to bf16's smallest: products with large gradients are
    exact where bf16 holds the value."""
    e = torch.arange(-126, 100, dtype=torch.float32)
    x = torch.exp2(e)[:, None].expand(-1, 32).contiguous()
    codes, scales = kept(oracle_lib, x)
    t = x.shape[0]
    dy = torch.zeros(t, t, device=DEV, dtype=torch.bfloat16)
    dy[torch.arange(t), torch.arange(t)] = 2.0
    dw = mps.act8_weight_grad(dy, codes, scales, torch.empty(t, 32, device=DEV), workspace(t, t, 32))
    assert torch.equal(dw.cpu(), x * 2)


@pytest.mark.parametrize("t,n,k", [(5000, 300, 200), (5000, 1024, 1040), (16384, 1024, 1024)])
def test_two_runs_give_the_same_bits(oracle_lib, t, n, k):
    g = gen(9)
    codes, scales = kept(oracle_lib, torch.randn(t, k, generator=g, device=DEV))
    dy = torch.randn(t, n, generator=g, device=DEV).to(torch.bfloat16)
    ws = workspace(t, n, k)
    runs = []
    for fill in (0, 255):
        ws.fill_(fill)  # whatever the workspace held
        runs.append(mps.act8_weight_grad(dy, codes, scales, torch.empty(n, k, device=DEV), ws).clone())
    assert torch.equal(*runs)


@pytest.mark.parametrize("dtype,t,n,k", [(torch.bfloat16, 40, 64, 64), (torch.float32, 40, 64, 64),
                                         (torch.bfloat16, 600, 4096, 4352), (torch.bfloat16, 257, 1024, 1024),
                                         (torch.float32, 1030, 4096, 4096)])
def test_offsets_past_32_bits(oracle_lib, dtype, t, n, k):
    """dy with more than 2^32 elements: a stride that puts the last tokens far out
    (in steps of less and of more than 2^25 elements)."""
    stride = (1 << 32) // (t - 4) // 8 * 8
    if t == 257:
        stride = (1 << 25) + 8
    g = gen(3)
    small = torch.randint(-8, 9, (t, n), generator=g, device=DEV).to(dtype)
    big = torch.empty(t * stride, dtype=dtype, device=DEV)
    dy = big.as_strided((t, n), (stride, 1))
    dy.copy_(small)
    x = torch.randint(-4, 5, (t, k), generator=g, device=DEV).float()
    codes, scales = kept(oracle_lib, x)
    dw = mps.act8_weight_grad(dy, codes, scales, torch.empty(n, k, device=DEV), workspace(t, n, k))
    assert torch.equal(dw, product(small, codes, scales, k)[0].float())


def test_refusals(oracle_lib):
    codes, scales = mps.act8_empty(5000, 64, DEV)
    dy = torch.zeros(5000, 8, device=DEV)
    dw = torch.zeros(8, 64, device=DEV)
    assert mps.act8_weight_grad_workspace_bytes(5000, 8, 64) > 0
    with pytest.raises(mps.MpsError, match="workspace"):
        mps.act8_weight_grad(dy, codes, scales, dw, None)
    with pytest.raises(mps.MpsError, match="too small"):
        mps.act8_weight_grad(dy, codes, scales, dw, torch.empty(256, dtype=torch.uint8, device=DEV))
    ws = workspace(5000, 8, 64)
    with pytest.raises(ValueError, match="codes"):
        mps.act8_weight_grad(dy, codes[:, :32], scales, dw, ws)
    with pytest.raises(ValueError, match="dw"):
        mps.act8_weight_grad(dy, codes, scales, dw[:7], ws)
    with pytest.raises(TypeError):
        mps.act8_weight_grad(dy.half(), codes, scales, dw, ws)
    with pytest.raises(ValueError, match="contiguous"):
        mps.act8_weight_grad(dy, codes, scales, torch.zeros(8, 128, device=DEV)[:, :64], ws)
