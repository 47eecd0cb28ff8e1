"""SwiGLU over 8-bit activations where the gate is far out: the sigmoid's own
relative error, made visible by a large up, down to where it counts as 0.

Bounds as in the tests of the operators: u = 2^-24, the sigmoid within 8 u (the
exponent's correction 2 u, the power 1 ulp, 1 + t one u, the reciprocal 1 ulp)
and 0 in place of anything below 2^-126."""
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref
from test_gpu_act8 import DEV, SIG, TYPES, frame_kept, gen, near, rounded
from train_reference import U

pytestmark = pytest.mark.gpu
UP = 1e30
NO_SIGMOID = 2.0 ** -126


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low,high", [(-87.25, -86.0), (-86.0, -80.0), (-80.0, -60.0), (-60.0, -1.0), (60.0, 130.0)])
def test_swiglu_of_a_gate_far_out(dtype, low, high):
    g = gen(int(high) + 200)
    gate = torch.empty(40, 1000, device=DEV).uniform_(low, high, generator=g).to(dtype).clamp(low, high)
    up = (UP * (1 + torch.rand(40, 1000, generator=g, device=DEV))).to(dtype)
    out = torch.empty_like(gate)
    mps.act8_swiglu(gate, up, out, *mps.act8_empty(40, 1000, DEV), *mps.act8_empty(40, 1000, DEV))
    want = ref.swiglu(gate.double(), up.double())
    near(out, want, rounded(want, dtype, SIG + 2 * U), "out")


@pytest.mark.parametrize("dtype", TYPES)
def test_swiglu_past_the_sigmoid_s_range(dtype):
    gate = torch.linspace(-200, -85, 4096, device=DEV).view(4, 1024).to(dtype)
    up = torch.full_like(gate, UP)
    out = torch.empty_like(gate)
    mps.act8_swiglu(gate, up, out, *mps.act8_empty(4, 1024, DEV), *mps.act8_empty(4, 1024, DEV))
    want = ref.swiglu(gate.double(), up.double())
    near(out, want, rounded(want, dtype, SIG + 2 * U) + (gate.double() * up.double()).abs() * NO_SIGMOID, "out")
    assert (out[gate < -89] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_swiglu_backward_of_a_gate_far_out(oracle_lib, dtype):
    """Kept gates next to the sigmoid's end are multiples of 8 (E4M3 under the run's
    scale): -80 within its range, -88 past it."""
    g = gen(3)
    gate = torch.tensor([-112.0, -104.0, -96.0, -88.0, -80.0, -72.0, 72.0, 80.0, 88.0, 96.0, 112.0], device=DEV)
    gate = gate[torch.randint(11, (20, 320), generator=g, device=DEV)]
    kg = [t.to(DEV) for t in ref.keep(oracle_lib, gate)]
    ku = [t.to(DEV) for t in ref.keep(oracle_lib, UP * (1 + torch.rand(20, 320, generator=g, device=DEV)))]
    dout = torch.randn(20, 320, generator=g, device=DEV).to(dtype)
    dgate, dup, again = torch.empty_like(dout), torch.empty_like(dout), frame_kept(20, 320)
    mps.act8_swiglu_backward(dout, *kg, *ku, dgate, dup, out_codes=again[0], out_scales=again[1])
    gd, ud, d = ref.values(*kg, 320).to(DEV), ref.values(*ku, 320).to(DEV), dout.double()
    assert torch.equal(gd.float(), gate)
    s = 1 / (1 + torch.exp(-gd))
    want_dg, want_du = ref.swiglu_backward(d, gd, ud)
    f = (1 + gd * (1 - s)).abs()
    size = (d * ud * s).abs() * ((SIG + 4 * U) * f + gd.abs() * (SIG * s + 2 * U * (1 - s)) + 2 * U)
    near(dgate, want_dg, rounded(want_dg, dtype, 0, size + (d * ud).abs() * (f + 1) * NO_SIGMOID), "dgate")
    near(dup, want_du, rounded(want_du, dtype, SIG + 2 * U, (d * gd).abs() * NO_SIGMOID), "dup")
