"""The attention block (FP8 projections, rotation, attention) as a training
step runs it: against float32 autograd of the same block on the unquantised
tensors, against its own calls made one by one, and captured into a graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.attention_block import AttentionBlock  # noqa: E402

HEADS, KV, D, HIDDEN = 4, 2, 128, 512
LENS = [200, 1, 130, 53]  # packed documents, 384 tokens


def make(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda shape, std: (torch.randn(shape, device="cuda", generator=gen) * std).to(torch.bfloat16)
    M = sum(LENS)
    cu = torch.tensor([0, 200, 201, 331, 384], dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(n) for n in LENS]).to(torch.int32).cuda()
    w_qkv, w_o = new(((HEADS + 2 * KV) * D, HIDDEN), 0.05), new((HIDDEN, HEADS * D), 0.05)
    block = AttentionBlock(w_qkv, w_o, HEADS, KV, M, cu, positions, bfp8.rope_table(256, D))
    block.quantize_weights()
    return block, new((M, HIDDEN), 1.0), new((M, HIDDEN), 1e-3)


def reference(block, x, dy):
    """The block in float32 by torch autograd, from its definition."""
    x, w_qkv, w_o = (t.float().detach().requires_grad_() for t in (x, block.w_qkv, block.w_o))
    qkv = (x @ w_qkv.t()).view(-1, HEADS + 2 * KV, D)
    cs = block.table[block.positions.long()][:, None]
    a, b = qkv[..., :D // 2], qkv[..., D // 2:]
    turned = torch.cat([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]], -1)
    q, k, v = turned[:, :HEADS], turned[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    out, at = [], 0
    for n in LENS:
        r = slice(at, at + n)
        s = torch.stack([q[r, h] @ k[r, h * KV // HEADS].t() for h in range(HEADS)]) / D ** 0.5
        s = s.masked_fill(torch.ones((n, n), device="cuda").triu(1).bool(), float("-inf"))
        p = torch.softmax(s, -1)
        out.append(torch.stack([p[h] @ v[r, h * KV // HEADS] for h in range(HEADS)], 1))
        at += n
    y = torch.cat(out).reshape(-1, HEADS * D) @ w_o.t()
    return (y,) + torch.autograd.grad((y * dy.float()).sum(), (x, w_qkv, w_o))


def test_block_matches_autograd():
    """Each FP8 linear is off by about 3.5 % of its output's norm (E4M3 keeps 4
    significant bits of either operand); forward chains two of them and backward
    four, errors that are independent: under 15 %.  A wrong head, position,
    sequence or sign is off by more than half."""
    block, x, dy = make()
    y = block.forward(x)
    got = (y,) + block.backward(dy)
    for name, a, b in zip(("y", "dx", "dw_qkv", "dw_o"), got, reference(block, x, dy)):
        err = ((a.float() - b).norm() / b.norm()).item()
        print(f"[block] {name}: {err:.4f}", flush=True)
        assert err < 0.15, (name, err)


def test_block_is_its_calls():
    """The in-place rotation, the fused rows and the shared workspaces change
    nothing: the same calls on tensors of their own give the same bytes."""
    block, x, dy = make(1)
    y = block.forward(x).clone()
    dx, dw_qkv, dw_o = (t.clone() for t in block.backward(dy))
    M = x.shape[0]
    (wq, ws), (oq, os_) = bfp8.quantize_weight_batch([block.w_qkv, block.w_o])
    xq, xs, xqt, xst = bfp8.quantize_act_dual(x)
    qkv = bfp8.gemm("NT", xq, xs, wq, ws, "act", "block").view(M, HEADS + 2 * KV, D)
    q, k, v = (t.contiguous() for t in (qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]))
    q, k = (bfp8.rope(t, block.table, block.positions) for t in (q, k))
    a, lse = bfp8.attention_forward(q, k, v, block.cu, block.cu)
    aq, as_, aqt, ast = bfp8.quantize_act_dual(a.view(M, -1))
    assert torch.equal(y, bfp8.gemm("NT", aq, as_, oq, os_, "act", "block"))
    dq_, ds_, dqt_, dst_ = bfp8.quantize_act_dual(dy)
    da = bfp8.gemm("NN", dq_, ds_, oq, os_, "act", "block").view(M, HEADS, D)
    assert torch.equal(dw_o, bfp8.gemm("NT", dqt_, dst_, aqt, ast, "act", "act"))
    dq, dk, dv = bfp8.attention_backward(da, q, k, v, a, lse, block.cu, block.cu)
    dq, dk = (bfp8.rope(t, block.table, block.positions, inverse=True) for t in (dq, dk))
    gq, gs, gqt, gst = bfp8.quantize_act_dual(torch.cat([dq, dk, dv], 1).view(M, -1))
    assert torch.equal(dx, bfp8.gemm("NN", gq, gs, wq, ws, "act", "block"))
    assert torch.equal(dw_qkv, bfp8.gemm("NT", gqt, gst, xqt, xst, "act", "act"))


def test_block_graph_replays_match_eager():
    block, x, dy = make(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x)
        block.backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    block.forward(x)
    block.backward(dy)
    names = ("y", "a", "lse", "dqkv", "dx", "dw_qkv", "dw_o")
    want = {n: block.buf[n].clone() for n in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x)
        block.backward(dy)
    torch.cuda.synchronize()
    eager = torch.randn((512, 512), device="cuda")
    for _ in range(3):
        for n in names:
            block.buf[n].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(block.buf[n], want[n]), n
        eager = eager @ eager.t() / 512
        torch.cuda.synchronize()


def test_block_refuses_sizes():
    w = torch.zeros((1024, 512), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((512, 512), dtype=torch.bfloat16, device="cuda")
    for args in ((w[:1000], o, 4, 2, 128), (w, o[:256], 4, 2, 128), (w, o, 4, 2, 100)):
        with pytest.raises(ValueError):
            AttentionBlock(*args, None, None, None)
