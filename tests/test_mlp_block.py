"""The feed-forward block (norm, FP8 projections, gated activation) as a training
step runs it, and a layer's two blocks with their gradients clipped: against
float32 autograd on the unquantised tensors, against their own calls made one by
one, and captured into a graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.attention_block import AttentionBlock  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.mlp_block import MLPBlock  # noqa: E402

HIDDEN, FFN, M = 512, 768, 384
BF = torch.bfloat16


def make(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda shape, std: (torch.randn(shape, device="cuda", generator=gen) * std).to(BF)
    w_norm = 1 + 0.1 * torch.randn(HIDDEN, device="cuda", generator=gen)
    block = MLPBlock(w_norm, new((2 * FFN, HIDDEN), 0.05), new((HIDDEN, FFN), 0.05), M)
    block.quantize_weights()
    return block, new((M, HIDDEN), 1.0), new((M, HIDDEN), 1.0), new((M, HIDDEN), 1e-3), \
        new((M, HIDDEN), 1e-3)


def mlp_reference(r, w_norm, w_gate_up, w_down, eps):
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + eps) * w_norm
    gate, up = (n @ w_gate_up.t()).split(w_down.shape[1], 1)
    return (gate * torch.sigmoid(gate) * up) @ w_down.t()


def reference(block, x, residual, dy, dr):
    """The block in float32 by torch autograd, from its definition."""
    r, w_norm, w_gate_up, w_down = (t.float().detach().requires_grad_() for t in (
        x.float() + residual.float(), block.w_norm, block.w_gate_up, block.w_down))
    y = mlp_reference(r, w_norm, w_gate_up, w_down, block.eps)
    grads = torch.autograd.grad((y * dy.float()).sum() + (r * dr.float()).sum(),
                                (r, w_gate_up, w_down, w_norm))
    return (y, r) + grads


def test_block_matches_autograd():
    """Each FP8 linear is off by about 3.5 % of its output's norm (E4M3 keeps 4
    significant bits of either operand); forward chains two of them and backward
    four, errors that are independent: under 15 %.  A wrong half, row, sum or sign
    is off by more than half."""
    block, x, residual, dy, dr = make()
    got = block.forward(x, residual) + block.backward(dy, dr)
    names = ("y", "r", "dx", "dw_gate_up", "dw_down", "dw_norm")
    for name, a, b in zip(names, got, reference(block, x, residual, dy, dr)):
        err = ((a.float() - b).norm() / b.norm()).item()
        print(f"[mlp] {name}: {err:.4f}", flush=True)
        assert err < (0.003 if name == "r" else 0.15), (name, err)


def test_block_is_its_calls():
    """The results that exist as codes only, the halves of fused rows and the shared
    workspace change nothing: the calls on tensors of their own, with the results
    in float32 and the package's quantisers between them, give the same bytes."""
    block, x, residual, dy, dr = make(1)
    y, r = (t.clone() for t in block.forward(x, residual))
    dx, dw_gate_up, dw_down, dw_norm = (t.clone() for t in block.backward(dy, dr))
    (gq, gs), (dq, ds) = bfp8.quantize_weight_batch([block.w_gate_up, block.w_down])
    assert torch.equal(r, (x.float() + residual.float()).to(BF))
    n32, _, rstd = bfp8.rmsnorm(r.float(), block.w_norm, eps=block.eps)
    nq, ns, nqt, nst = bfp8.quantize_act_dual(n32)
    gate_up = bfp8.gemm("NT", nq, ns, gq, gs, "act", "block")
    gate, up = (t.contiguous() for t in gate_up.split(FFN, 1))
    hq, hs, hqt, hst = bfp8.quantize_act_dual(bfp8.swiglu(gate.float(), up.float()))
    assert torch.equal(y, bfp8.gemm("NT", hq, hs, dq, ds, "act", "block"))
    yq, ys, yqt, yst = bfp8.quantize_act_dual(dy)
    dh = bfp8.gemm("NN", yq, ys, dq, ds, "act", "block")
    assert torch.equal(dw_down, bfp8.gemm("NT", yqt, yst, hqt, hst, "act", "act"))
    d32 = torch.cat(bfp8.swiglu_backward(dh.float(), gate.float(), up.float()), 1)
    uq, us, uqt, ust = bfp8.quantize_act_dual(d32)
    dn = bfp8.gemm("NN", uq, us, gq, gs, "act", "block")
    assert torch.equal(dw_gate_up, bfp8.gemm("NT", uqt, ust, nqt, nst, "act", "act"))
    for a, b in zip((dx, dw_norm), bfp8.rmsnorm_backward(dn, r, block.w_norm, rstd, dr)):
        assert torch.equal(a, b)


def layer(seed=2, tokens=M):
    """A pre-norm layer on a residual stream, the last rows of its micro-batch unused,
    and the clipping of all its weights' gradients."""
    mlp, x, residual, dy, dr = make(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 50)
    new = lambda shape, std: (torch.randn(shape, device="cuda", generator=gen) * std).to(BF)
    cu = torch.tensor([0, 100, tokens], dtype=torch.int32, device="cuda")
    positions = torch.full((M,), -1, dtype=torch.int32)
    positions[:tokens] = torch.cat([torch.arange(100), torch.arange(tokens - 100)])
    attn = AttentionBlock(new((8 * 128, HIDDEN), 0.05), new((HIDDEN, 4 * 128), 0.05), 4, 2, M, cu,
                          positions.cuda(), bfp8.rope_table(384, 128),
                          w_norm=1 + 0.1 * torch.randn(HIDDEN, device="cuda", generator=gen))
    attn.quantize_weights()
    b, c = attn.buf, mlp.buf
    grads = [b["dw_qkv"], b["dw_o"], b["dw_norm"], c["dw_gate_up"], c["dw_down"], c["dw_norm"]]
    clip = bfp8.GradClip(grads, [torch.empty_like(g) for g in grads])

    def step():
        y1, r1 = attn.forward(x, residual)
        y2, r2 = mlp.forward(y1, r1)
        d1, *_ = mlp.backward(dy, dr)
        d0, *_ = attn.backward(d1, d1)  # dx is the gradient of x and of the residual alike
        norm = clip.clip(0.01)
        return [y2, r2, d1, d0, norm, *clip.out]
    return step, clip, attn, mlp, (x, residual, dy, dr)


def test_a_layer_matches_autograd():
    """Four FP8 linears forward and eight in all, the attention's and the residual
    streams' bf16 roundings beside them: each quantity has at most eight FP8
    products of 3.5 % on its way, independent: under 15 %."""
    step, clip, attn, mlp, (x, residual, dy, dr) = layer()
    y2, r2, _, d0, _, *_ = step()
    leaves = [t.float().detach().requires_grad_() for t in (
        x.float() + residual.float(), attn.w_norm, attn.w_qkv, attn.w_o, mlp.w_norm, mlp.w_gate_up,
        mlp.w_down)]
    r0, wn1, w_qkv, w_o, wn2, wgu, wd = leaves
    n = r0 * torch.rsqrt((r0 * r0).mean(1, keepdim=True) + attn.eps) * wn1
    qkv = (n @ w_qkv.t()).view(M, 8, 128)
    cs = attn.table[attn.positions.long()][:, None]
    a, b = qkv[..., :64], qkv[..., 64:]
    turned = torch.cat([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]], -1)
    out = []
    for lo, hi in ((0, 100), (100, M)):
        heads = []
        for h in range(4):
            s = turned[lo:hi, h] @ turned[lo:hi, 4 + h // 2].t() / 128 ** 0.5
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), float("-inf"))
            heads.append(torch.softmax(s, -1) @ qkv[lo:hi, 6 + h // 2])
        out.append(torch.stack(heads, 1))
    r1 = r0 + torch.cat(out).reshape(M, -1) @ w_o.t()
    y = mlp_reference(r1, wn2, wgu, wd, mlp.eps)
    loss = (y * dy.float()).sum() + (r1 * dr.float()).sum()
    want = torch.autograd.grad(loss, leaves)
    got = [d0, *(attn.buf[k] for k in ("dw_norm", "dw_qkv", "dw_o")),
           *(mlp.buf[k] for k in ("dw_norm", "dw_gate_up", "dw_down"))]
    for name, p, q in zip(("y", "r", "dx", "dw_norm", "dw_qkv", "dw_o", "dw_norm2", "dw_gate_up", "dw_down"),
                          [y2, r2] + got, [y, r1] + list(want)):
        err = ((p.float() - q).norm() / q.norm()).item()
        print(f"[layer] {name}: {err:.4f}", flush=True)
        assert err < 0.15, (name, err)


def test_an_attention_block_with_a_norm_is_its_calls():
    _, _, attn, _, (x, residual, dy, dr) = layer(3)
    y, r = (t.clone() for t in attn.forward(x, residual))
    dx, dw_qkv, dw_o, dw_norm = (t.clone() for t in attn.backward(dy, dr))
    plain = AttentionBlock(attn.w_qkv, attn.w_o, 4, 2, M, attn.cu, attn.positions, attn.table)
    plain.quantize_weights()
    n, r2, rstd = bfp8.rmsnorm(x, attn.w_norm, residual, eps=attn.eps)
    assert torch.equal(r, r2)
    # from the norm in float32: the codes of the block's QKV input
    n32, _, _ = bfp8.rmsnorm(r.float(), attn.w_norm, eps=attn.eps)
    for a, b in zip(bfp8.quantize_act_dual_kmajor(n32), (attn.buf[k] for k in ("xq", "xs", "xqt", "xst"))):
        assert torch.equal(a, b)
    # the rest is the block without a norm: the QKV rows of the same codes, and its
    # backward pass from the same buffers
    qkv = bfp8.gemm("NT", *(attn.buf[k] for k in ("xq", "xs", "wqkv_q", "wqkv_s")), "act_km", "block")
    bfp8.rope(qkv.view(M, 8, 128)[:, :6], attn.table, attn.positions, out=qkv.view(M, 8, 128)[:, :6])
    assert torch.equal(qkv.view(M, 8, 128), attn.buf["qkv"])
    plain.forward(x)
    for k in ("xqt", "xst", "qkv", "a", "lse", "aqt", "ast"):
        plain.buf[k].copy_(attn.buf[k])
    dn, dw_qkv2, dw_o2 = plain.backward(dy)
    assert torch.equal(dw_qkv, dw_qkv2) and torch.equal(dw_o, dw_o2) and torch.equal(dn, attn.buf["dn"])
    for a, b in zip((dx, dw_norm), bfp8.rmsnorm_backward(dn, r, attn.w_norm, rstd, dr)):
        assert torch.equal(a, b)


def test_a_layers_clipped_gradients():
    step, clip, *_ = layer()
    norm = step()[4]
    total = bfp8.grad_norm(clip.out)
    assert norm > 0.01
    # each clipped bf16 value is off by 2^-8 of itself at most: so is their norm
    assert abs(total.item() - 0.01) <= 0.01 * (2.0 ** -8 + 2.0 ** -20)


@pytest.mark.parametrize("tokens", [M, 300])
def test_a_layers_step_in_a_graph(tokens):
    """Captured, and replayed with eager work between: the eager bytes."""
    step, *_ = layer(7, tokens)
    want = [t.clone() for t in step()]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)


def test_refusals():
    block, x, residual, dy, dr = make()
    with pytest.raises(RuntimeError, match="forward"):
        block.backward(dy, dr)
    fresh = MLPBlock(block.w_norm, block.w_gate_up, block.w_down, M)
    with pytest.raises(RuntimeError, match="quantize_weights"):
        fresh.forward(x, residual)
    for bad in (x[:256], x.float(), x.cpu()):
        with pytest.raises(ValueError):
            block.forward(bad, residual)
        with pytest.raises(ValueError):
            block.forward(x, bad)
    _, _, attn, _, _ = layer()
    for call in (lambda: attn.forward(x), lambda: attn.backward(dy),
                 lambda: attn.forward(x, residual[:256])):
        with pytest.raises(ValueError):
            call()
    plain = AttentionBlock(attn.w_qkv, attn.w_o, 4, 2, M, attn.cu, attn.positions, attn.table)
    with pytest.raises(ValueError, match="only with one"):
        plain.forward(x, residual)
    with pytest.raises(ValueError, match="w_norm"):
        AttentionBlock(attn.w_qkv, attn.w_o, 4, 2, M, attn.cu, attn.positions, attn.table,
                       w_norm=attn.w_norm[:256])
