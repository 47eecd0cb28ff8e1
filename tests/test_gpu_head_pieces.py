"""linear_cross_entropy where its g is several pieces of the vocabulary and many
tiles of tokens take part in each: weights that are read as they lie and packed,
both types, dweight written and added to."""
import pytest
import torch

import head_precision as hp
import mixed_precision_sharded_amd as mps
import model_reference as ref
from test_gpu_head import check, problem
from test_gpu_head_precision import gradients

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32

# tokens, vocabulary, features, type: three pieces each, the first of them a short one.
SIZES = [(2600, 240007, 64, BF16), (300, 130001, 4104, BF16), (700, 100003, 1000, F32)]


@pytest.mark.parametrize("tokens,vocab,cols,dtype", SIZES)
def test_many_rows_in_every_piece(tokens, vocab, cols, dtype):
    p = problem(tokens, vocab, cols, dtype)
    p[3].div_(tokens)
    assert int(ref.live_rows(p[2], p[3], vocab).sum()) > (2048 if tokens > 2048 else 200)
    first = check(*p, dw_type=F32)
    again = check(*p, dw_type=F32)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    before = torch.randn(vocab, cols, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(dtype)
    check(*p, before=before)
    del first, again, before
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens,vocab,cols,dtype", [s for s in SIZES if s[3] == BF16])
@pytest.mark.parametrize("gap", [0.0, 24.0])
def test_g_of_every_piece(tokens, vocab, cols, dtype, gap):
    """The label's 16 bits, and what lies far below it, whether a piece's exponentials stayed or its logits were made again."""
    p = hp.problem(tokens, vocab, cols, gap, device=DEV)
    r = hp.exact(*p)
    dh, dw = gradients(*p, F32)
    assert hp.outside(dw, r["dw"], r["dw_off"]) == 0
    assert hp.outside(dh, r["dh"], r["dh_off"]) == 0
    del r, dh, dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens,vocab,cols,dtype", SIZES)
def test_pieces_replayed(tokens, vocab, cols, dtype):
    """Captured, and replayed with other inputs and the program's own work between: the same bits as the call itself."""
    p, q = problem(tokens, vocab, cols, dtype), problem(tokens, vocab, cols, dtype, seed=9)
    ws = torch.empty(mps.linear_cross_entropy_workspace_bytes(tokens, vocab, cols, dtype), dtype=torch.uint8, device=DEV)
    loss, dh, dw = torch.empty(1, device=DEV), torch.empty_like(p[0]), torch.empty_like(p[1])
    eager = []
    for inputs in (p, q):
        mps.linear_cross_entropy(*inputs, loss, ws, dhidden=dh, dweight=dw)
        eager.append((loss.clone(), dh.clone(), dw.clone()))
    held = [x.clone() for x in p]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mps.linear_cross_entropy(*held, loss, ws, dhidden=dh, dweight=dw)
    for inputs, want in ((q, eager[1]), (p, eager[0]), (q, eager[1])):
        for a, b in zip(held, inputs):
            a.copy_(b)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, dh, dw), want):
            assert torch.equal(a, b)
    del eager, held, graph
    torch.cuda.empty_cache()
