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


def layer(seed=2):
    """An attention block and a feed-forward block on one residual stream, and the
    clipping of all their weights' gradients."""
    mlp, x, residual, dy, dr = make(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 50)
    new = lambda shape, std: (torch.randn(shape, device="cuda", generator=gen) * std).to(BF)
    cu = torch.tensor([0, 100, 384], dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(100), torch.arange(284)]).to(torch.int32).cuda()
    attn = AttentionBlock(new((8 * 128, HIDDEN), 0.05), new((HIDDEN, 4 * 128), 0.05), 4, 2, M, cu,
                          positions, bfp8.rope_table(384, 128))
    attn.quantize_weights()
    b, c = attn.buf, mlp.buf
    clip = bfp8.GradClip([b["dw_qkv"], b["dw_o"], c["dw_gate_up"], c["dw_down"], c["dw_norm"]])

    def step():
        a = attn.forward(x)
        y, r = mlp.forward(a, x)
        dx, *_ = mlp.backward(dy, dr)
        attn.backward(dx)
        norm = clip.clip(0.01)
        return [y, r, dx, norm, *clip.out]
    return step, clip


def test_a_layers_step_and_its_clipped_gradients():
    step, clip = layer()
    *_, norm = step()[:4]
    total = bfp8.grad_norm(clip.out)
    assert norm > 0.01
    # each clipped bf16 value is off by 2^-8 of itself at most: so is their norm
    assert abs(total.item() - 0.01) <= 0.01 * (2.0 ** -8 + 2.0 ** -20)


def test_a_layers_step_in_a_graph():
    """Captured, and replayed with eager work between: the eager bytes."""
    step, _ = layer(7)
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
