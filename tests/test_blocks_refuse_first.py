"""The blocks with a norm: gradients and streams of another type or with other strides are
refused before anything is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.attention_block import AttentionBlock  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.mlp_block import MLPBlock  # noqa: E402

BF = torch.bfloat16


def test_refused_before_a_result_is_touched():
    M = hidden = 256
    new = lambda *s: (torch.randn(s, device="cuda") * 0.1).to(BF)
    cu = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    block = AttentionBlock(new(4 * 128, hidden), new(hidden, 2 * 128), 2, 1, M, cu,
                           torch.arange(M, dtype=torch.int32, device="cuda"), bfp8.rope_table(M, 128),
                           w_norm=torch.ones(hidden, device="cuda"))
    mlp = MLPBlock(torch.ones(hidden, device="cuda"), new(2 * 128, hidden), new(hidden, 128), M)
    x, residual, dy, dr = (new(M, hidden) for _ in range(4))
    for b, names in ((block, ("y", "r", "rstd", "dx", "dw_qkv", "dw_o", "dw_norm")),
                     (mlp, ("y", "r", "rstd", "dx", "dw_gate_up", "dw_down", "dw_norm"))):
        b.quantize_weights()
        b.forward(x, residual)
        b.backward(dy, dr)
        before = {n: b.buf[n].clone() for n in names}
        for call in (lambda: b.backward(2 * dy, dr.float()), lambda: b.backward(2 * dy, dr.half()),
                     lambda: b.backward(2 * dy, dr.t()), lambda: b.forward(2 * x, residual.float()),
                     lambda: b.forward(2 * x, residual.t()),
                     lambda: b.forward(2 * x.float(), residual.float())):
            with pytest.raises(ValueError):
                call()
            for n in names:
                assert torch.equal(b.buf[n], before[n]), n
