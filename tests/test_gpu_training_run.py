"""The operators together, as a training step uses them: a gated MLP block and
a head under the policy loss, backward from 8-bit activations into the fp32
gradients of the step's list, the clipped step; against the 64-bit forms on
the same kept bytes, and the step against the oracle.  Then the same run in a
captured graph, on other streams, and at the same time on two."""
import numpy as np
import pytest
import torch

import mixed_precision_sharded_amd as mps
import train_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROWS, DIM, FFN, VOCAB = 200, 264, 488, 1007
EPS = 1e-5


class Block:
    """One micro-batch's buffers, and the calls of its forward and backward pass."""

    def __init__(self, seed, rows=ROWS):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s, scale=1.0, dtype=torch.bfloat16: (torch.randn(*s, generator=g, device=DEV) * scale).to(dtype)  # noqa: E731
        e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        f32 = torch.float32
        self.rows = rows
        self.h = r(rows, DIM)
        self.w_norm = 1 + r(DIM, scale=0.1, dtype=f32)
        self.w_in, self.w_down, self.w_head = r(2 * FFN, DIM, scale=0.06), r(DIM, FFN, scale=0.05), r(VOCAB, DIM, scale=0.1)
        self.labels = torch.randint(VOCAB, (rows,), generator=g, device=DEV)
        self.labels[::7] = -100
        self.old, self.ref = r(rows, scale=0.3, dtype=f32) - 7, r(rows, scale=0.3, dtype=f32) - 7
        self.adv, self.weight = r(rows, dtype=f32), torch.full((rows,), 1.0 / rows, device=DEV)
        self.y, self.rstd = e(rows, DIM), e(rows, dtype=f32)
        self.both, self.act, self.o = e(rows, 2 * FFN), e(rows, FFN), e(rows, DIM)
        self.logits, self.loss = e(rows, VOCAB), e(1, dtype=f32)
        self.x8, self.g8, self.u8, self.o8 = (mps.act8_empty(rows, c, DEV) for c in (DIM, FFN, FFN, DIM))
        self.y8, self.a8 = mps.act8_empty(rows, DIM, DEV), mps.act8_empty(rows, FFN, DEV)
        self.do, self.da, self.dboth, self.dy, self.dh = e(rows, DIM), e(rows, FFN), e(rows, 2 * FFN), e(rows, DIM), e(rows, DIM)
        shapes = {"norm": (DIM,), "in": (2 * FFN, DIM), "down": (DIM, FFN), "head": (VOCAB, DIM)}
        self.grads = {k: e(*s, dtype=f32) for k, s in shapes.items()}
        need = max(mps.policy_loss_workspace_bytes(rows, VOCAB), mps.act8_rmsnorm_backward_workspace_bytes(rows, DIM),
                   *(mps.act8_weight_grad_workspace_bytes(rows, *s) for k, s in shapes.items() if k != "norm"))
        self.ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)

    def run(self, accumulate=False, stream=None):
        kw = dict(stream=stream)
        mps.act8_rmsnorm(self.h, self.w_norm, EPS, self.y, self.rstd, *self.x8, **kw)
        torch.mm(self.y, self.w_in.t(), out=self.both)
        mps.act8_swiglu(self.both[:, :FFN], self.both[:, FFN:], self.act, *self.g8, *self.u8, **kw)
        torch.mm(self.act, self.w_down.t(), out=self.o)
        self.o += self.h
        mps.act8_save(self.o, *self.o8, **kw)
        torch.mm(self.o, self.w_head.t(), out=self.logits)
        # The gradient of the logits in their own memory.
        mps.policy_loss(self.logits, self.labels, self.old, self.adv, self.weight, self.loss, self.ws, clip_low=0.2,
                        clip_high=0.28, ref_logp=self.ref, kl_coef=0.05, dlogits=self.logits, **kw)
        mps.act8_weight_grad(self.logits, *self.o8, self.grads["head"], self.ws, accumulate=accumulate, **kw)
        torch.mm(self.logits, self.w_head, out=self.do)
        torch.mm(self.do, self.w_down, out=self.da)
        mps.act8_swiglu_backward(self.da, *self.g8, *self.u8, self.dboth[:, :FFN], self.dboth[:, FFN:], *self.a8, **kw)
        mps.act8_weight_grad(self.do, *self.a8, self.grads["down"], self.ws, accumulate=accumulate, **kw)
        torch.mm(self.dboth, self.w_in, out=self.dy)
        mps.act8_rmsnorm_backward(self.dy, *self.x8, self.rstd, self.w_norm, self.dh, self.grads["norm"], self.ws,
                                  residual_grad=self.do, accumulate=accumulate, out_codes=self.y8[0], out_scales=self.y8[1], **kw)
        mps.act8_weight_grad(self.dboth, *self.y8, self.grads["in"], self.ws, accumulate=accumulate, **kw)

    def outputs(self):
        return [self.loss, self.logits, self.dh, *self.grads.values(), *self.x8, *self.g8, *self.u8, *self.o8, *self.y8, *self.a8]


def clones(b):
    return [t.clone() for t in b.outputs()]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_against_the_formulas(oracle_lib):
    b = Block(1)
    b.run()
    v = lambda kept, cols: ref.values(*kept, cols).to(DEV)  # noqa: E731
    # Each operator on the very inputs it had, in 64 bits; bf16 tensors between them as they were handed on.
    for kept, x in ((b.x8, b.h), (b.g8, b.both[:, :FFN]), (b.u8, b.both[:, FFN:]), (b.o8, b.o)):
        codes, scales = ref.keep(oracle_lib, x)
        assert torch.equal(kept[0].cpu(), codes) and torch.equal(kept[1].cpu(), scales)
    # b.logits holds the gradient now; the logits again, with the same product of the same operands.
    p = ref.policy(torch.mm(b.o, b.w_head.t()), b.labels, b.old, b.adv, b.weight, 0.2, 0.28, b.ref, 0.05)
    assert abs(b.loss.item() - p["loss"].item()) <= 1e-5 * p["row_loss"].abs().sum().item()
    near = lambda got, want, tol: (got.double() - want).norm() <= tol * want.norm()  # noqa: E731
    half = 2.0 ** -8  # one rounding to bf16, at most
    assert near(b.logits, p["dlogits"], half)
    dg, du = ref.swiglu_backward(b.da.double(), v(b.g8, FFN), v(b.u8, FFN))
    assert near(b.dboth, torch.cat([dg, du], 1), half)
    dh, dw, y = ref.rmsnorm_backward(b.dy.double(), v(b.x8, DIM), b.rstd.double(), b.w_norm.double(), b.do.double())
    assert near(b.dh, dh, half) and near(b.grads["norm"], dw, 2e-6)
    # fp32 sums of exact products: far below one bf16 rounding.
    for name, d, kept, k in (("head", b.logits, b.o8, DIM), ("down", b.do, b.a8, FFN), ("in", b.dboth, b.y8, DIM)):
        assert near(b.grads[name], torch.mm(d.double().t().contiguous(), v(kept, k).contiguous()), 2e-6), name
    # And the whole against the gradients without any 8-bit rounding: E4M3 keeps 4 bits, an error of at most 2^-4
    # of a value, of random sign; its mean square over a binade is below (2^-5)^2, and a gradient is linear in it
    # to first order through at most three kept factors.
    leaves = [t.double().requires_grad_() for t in (b.w_norm, b.w_in, b.w_down, b.w_head)]
    h = b.h.double()
    yy, _ = ref.rmsnorm(h, leaves[0], EPS)
    z = yy @ leaves[1].t()
    o = ref.swiglu(z[:, :FFN], z[:, FFN:]) @ leaves[2].t() + h
    ref.policy(o @ leaves[3].t(), b.labels, b.old, b.adv, b.weight, 0.2, 0.28, b.ref, 0.05)["loss"].backward()
    for name, leaf in zip(("norm", "in", "down", "head"), leaves):
        assert near(b.grads[name], leaf.grad, 0.12), name


def test_two_micro_batches_and_the_clipped_step(oracle_lib):
    """Gradients accumulate over micro-batches in the step's own buffers."""
    b = Block(2)
    b.run()
    first = {k: v.clone() for k, v in b.grads.items()}
    b.run(accumulate=True)
    for k, g in b.grads.items():
        assert torch.equal(g, first[k] * 2), k  # the same batch twice: doubling is exact
    names = ["norm", "in", "down", "head"]
    grads = [b.grads[k] for k in names]
    masters = [t.float().clone() for t in (b.w_norm, b.w_in, b.w_down, b.w_head)]
    m, v = [torch.zeros_like(t) for t in masters], [torch.zeros_like(t) for t in masters]
    host = [[t.cpu().numpy().reshape(-1).copy() for t in col] for col in (masters, m, v, grads)]
    tl = mps.TensorList(masters, m, v, grads)
    step = torch.zeros(1, dtype=torch.int32, device=DEV)
    coef = torch.zeros(1, device=DEV)
    mps.adamw_clipped_step(tl, step, 3e-4, 0.9, 0.95, 1e-8, 0.1, max_norm=1.0, grad_scale=0.5, coef_out=coef)
    c = np.float32(coef.item())
    for i in range(len(names)):
        oracle_lib.adamw_step(host[0][i], host[1][i], host[2][i], host[3][i], None, c, 1, 3e-4, 0.9, 0.95, 1e-8, 0.1)
        assert np.array_equal(masters[i].cpu().numpy().reshape(-1), host[0][i]), names[i]


def test_captured_and_replayed():
    """Captured on its first call; each replay equals the eager run, with eager
    work and other inputs between replays."""
    b, other = Block(3), Block(4)
    b.run()
    want = clones(b)
    for t in b.outputs():
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()  # the library calls between the operators load their kernels before the capture
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        b.run()
    for i in range(3):
        for t in b.outputs():
            t.fill_(i)
        graph.replay()
        other.run()
        torch.cuda.synchronize()
        assert same(b.outputs(), want), i
    h = b.h.clone()
    b.h.copy_(other.h)
    graph.replay()
    changed = clones(b)
    b.run()
    assert same(b.outputs(), changed) and not same(changed, want)
    b.h.copy_(h)
    graph.replay()
    assert same(b.outputs(), want)


def test_capture_needs_no_earlier_call():
    """Each operator alone in a graph, new sizes, nothing before it."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(37, 135, generator=g, device=DEV)
    codes, scales = mps.act8_empty(37, 135, DEV)
    dw = torch.empty(135, 135, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mps.act8_save(x, codes, scales)
        mps.act8_load(codes, scales, out)
        mps.act8_weight_grad(x, codes, scales, dw, ws)
    for _ in range(3):
        codes.zero_(), dw.zero_(), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c, s = mps.act8_empty(37, 135, DEV)
        mps.act8_save(x, c, s)
        assert torch.equal(c, codes) and torch.equal(s, scales)
        assert torch.equal(mps.act8_load(c, s, torch.empty_like(x)), out)
        assert torch.equal(mps.act8_weight_grad(x, c, s, torch.empty_like(dw), ws), dw)


def test_two_streams_at_once():
    """Two blocks with buffers and workspaces of their own, on two streams."""
    blocks = [Block(6), Block(7, rows=333)]
    want = []
    for b in blocks:
        b.run()
        want.append(clones(b))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for b in blocks:
            for t in b.outputs():
                t.zero_()
        torch.cuda.synchronize()
        for s, b in zip(streams, blocks):
            with torch.cuda.stream(s):
                b.run()
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert same(b.outputs(), w)


def test_the_stream_argument():
    """stream= enqueues there, behind what that stream has to do first."""
    s = torch.cuda.Stream()
    x = torch.randn(4000, 4096, device=DEV)
    codes, scales = mps.act8_empty(4000, 4096, DEV)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = x
        for _ in range(20):
            y = y * 1.5 - 0.25
    mps.act8_save(y, codes, scales, stream=s)
    mps.act8_load(codes, scales, out, stream=s)
    s.synchronize()
    c, k = mps.act8_empty(4000, 4096, DEV)
    mps.act8_save(y, c, k)
    assert torch.equal(c, codes) and torch.equal(mps.act8_load(c, k, torch.empty_like(x)), out)
