"""The 64-bit plain forms against differences of their own forward functions
(CPU): what the GPU tests compare with has the gradients of what it computes."""
import pytest
import torch

import train_reference as ref


def slope_of(f, x, h):
    """df/dx by central differences, f a scalar function of a matrix."""
    out = torch.empty_like(x)
    flat = x.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        a = f(x)
        flat[i] = keep - h
        b = f(x)
        flat[i] = keep
        out.view(-1)[i] = (a - b) / (2 * h)
    return out


def gen(seed):
    return torch.Generator().manual_seed(seed)


# Central differences of step h: h^2 / 6 of a third derivative of order one,
# and 2^-53 / h of rounding, both far below 1e-7 at h = 1e-5.
H, NEAR = 1e-5, 1e-7


def test_rmsnorm_gradient_is_the_slope():
    g = gen(1)
    x, w, dy = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(3))
    w = w[0]
    res = torch.randn(3, 7, generator=g, dtype=torch.float64)
    _, r = ref.rmsnorm(x, w, 1e-12)
    dx, dw, y = ref.rmsnorm_backward(dy, x, r, w, res)
    f = lambda x_, w_: (ref.rmsnorm(x_, w_, 1e-12)[0] * dy).sum()  # noqa: E731
    assert torch.allclose(dx - res, slope_of(lambda t: f(t, w), x.clone(), H), atol=NEAR)
    assert torch.allclose(dw, slope_of(lambda t: f(x, t[0]), w[None].clone(), H)[0], atol=NEAR)
    assert torch.allclose(y, ref.rmsnorm(x, w, 1e-12)[0])


def test_swiglu_gradient_is_the_slope():
    g = gen(2)
    gate, up, d = (torch.randn(4, 5, generator=g, dtype=torch.float64) * 2 for _ in range(3))
    dg, du = ref.swiglu_backward(d, gate, up)
    assert torch.allclose(dg, slope_of(lambda t: (ref.swiglu(t, up) * d).sum(), gate.clone(), H), atol=NEAR)
    assert torch.allclose(du, slope_of(lambda t: (ref.swiglu(gate, t) * d).sum(), up.clone(), H), atol=NEAR)


@pytest.mark.parametrize("with_ref", [False, True])
def test_policy_gradient_is_the_slope(with_ref):
    g = gen(3)
    rows, vocab = 12, 9
    x = torch.randn(rows, vocab, generator=g, dtype=torch.float64)
    labels = torch.randint(vocab, (rows,), generator=g)
    labels[3] = -100
    adv = torch.randn(rows, generator=g)
    adv[5] = 0
    weight = torch.rand(rows, generator=g)
    weight[7] = 0
    logp = torch.log_softmax(x, 1)[torch.arange(rows), labels.clamp(min=0)]
    # Ratios on both sides of the clip, none within 0.01 of its borders.
    old = (logp - torch.tensor([0.0, 0.5, -0.5, 0.1] * 3)).float()
    kl = dict(ref=(logp + 0.3).float(), kl_coef=0.1) if with_ref else {}
    f = lambda t: ref.policy(t, labels, old, adv, weight, 0.2, 0.3, **kl)["loss"]  # noqa: E731
    got = ref.policy(x, labels, old, adv, weight, 0.2, 0.3, **kl)
    assert torch.allclose(got["dlogits"], slope_of(f, x.clone(), H), atol=NEAR)
    assert not got["dlogits"][3].any() and not got["dlogits"][7].any()
    if not with_ref:
        assert (got["slope"][got["live"]] == 0).sum() > 1  # some rows are on the clip's flat side


def test_keep_is_the_rule(oracle_lib):
    """Codes and scales of the oracle read back within half a step of the
    largest code's grid, and exactly where the values are codes already."""
    g = gen(4)
    x = torch.randn(5, 70, generator=g) * torch.tensor([1e-30, 1e-3, 1.0, 1e3, 1e30])[:, None]
    codes, scales = ref.keep(oracle_lib, x)
    assert codes.shape == (5, 96) and scales.shape == (5, 3)
    v = ref.values(codes, scales, 70)
    runs = torch.nn.functional.pad(x.double(), (0, 26)).view(5, 3, 32).abs().amax(2).repeat_interleave(32, 1)[:, :70]
    # E4M3 keeps 4 bits: half a step is 2^-4 of a value, and at most 2^-10 of 448's power of two below.
    assert ((v - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, runs * 2.0 ** -17)).all()
    again, s2 = ref.keep(oracle_lib, v.float())
    assert torch.equal(ref.values(again, s2, 70), v)
    assert not codes[:, 70:].any()
