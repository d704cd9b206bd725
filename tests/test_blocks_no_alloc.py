"""The layer's blocks allocate nothing in a pass: their buffers and the workspaces of all
their calls are made with them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.attention_block import AttentionBlock  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.mlp_block import MLPBlock  # noqa: E402

BF = torch.bfloat16


def new(*shape, std=1.0):
    return (torch.randn(shape, device="cuda") * std).to(BF)


def mlp(tokens, hidden, ffn):
    block = MLPBlock(torch.ones(hidden, device="cuda"), new(2 * ffn, hidden, std=0.02),
                     new(hidden, ffn, std=0.02), tokens)
    x, residual, dy, dr = (new(tokens, hidden) for _ in range(4))
    return block, lambda: block.forward(x, residual), lambda: block.backward(dy, dr)


def attention(tokens, hidden, heads, kv_heads, norm):
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    block = AttentionBlock(new((heads + 2 * kv_heads) * 128, hidden, std=0.02), new(hidden, heads * 128, std=0.02),
                           heads, kv_heads, tokens, cu, torch.arange(tokens, dtype=torch.int32, device="cuda"),
                           bfp8.rope_table(tokens, 128),
                           w_norm=torch.ones(hidden, device="cuda") if norm else None)
    x, residual, dy, dr = (new(tokens, hidden) for _ in range(4))
    if not norm:
        residual = dr = None
    return block, lambda: block.forward(x, residual), lambda: block.backward(dy, dr)


CASES = [(mlp, 128, 2048, 6144), (mlp, 2048, 2048, 6144), (mlp, 4096, 2048, 6144), (mlp, 384, 512, 768)] + \
    [(attention, tokens, 2048, 16, 8, norm) for tokens in (128, 1024, 4096) for norm in (False, True)] + \
    [(attention, 4096, 4096, 32, 8, False)]


@pytest.mark.parametrize("make,sizes", [(c[0], c[1:]) for c in CASES])
def test_a_pass_allocates_nothing(make, sizes):
    block, forward, backward = make(*sizes)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]
    block.quantize_weights()
    first = count()
    forward()
    backward()
    assert count() - first == 0, "a first pass"
    for _ in range(2):
        forward()
        backward()
    torch.cuda.synchronize()
    assert count() - first == 0
