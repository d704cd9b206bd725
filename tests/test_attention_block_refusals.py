"""What the attention block refuses before it enqueues anything."""
import pytest
import torch

import test_attention_block as base

pytestmark = pytest.mark.gpu


def test_rows_of_another_size():
    """x and dy of more rows or columns than the block has would be quantised
    past the ends of its buffers."""
    block, x, dy = base.make()
    block.forward(x)
    M, hidden = x.shape
    for shape in ((M + 128, hidden), (M - 128, hidden), (M, hidden + 128), (M, hidden // 2),
                  (M * hidden,), (1, M, hidden)):
        t = torch.zeros(shape, dtype=x.dtype, device="cuda")
        with pytest.raises(ValueError, match="x must be"):
            block.forward(t)
        with pytest.raises(ValueError, match="dy must be"):
            block.backward(t)
    with pytest.raises(ValueError, match="x must be"):
        block.forward(x.cpu())
    with pytest.raises(ValueError, match="dy must be"):
        block.backward(dy.cpu())


def test_steps_out_of_order():
    """Without codes of the weights, or a forward pass, the buffers hold nothing."""
    block, x, dy = base.make()
    fresh = base.AttentionBlock(block.w_qkv, block.w_o, base.HEADS, base.KV, x.shape[0], block.cu,
                                block.positions, block.table)
    with pytest.raises(RuntimeError, match="quantize_weights"):
        fresh.forward(x)
    with pytest.raises(RuntimeError, match="forward"):
        fresh.backward(dy)
    fresh.quantize_weights()
    with pytest.raises(RuntimeError, match="forward"):
        fresh.backward(dy)
    want = [block.forward(x), *block.backward(dy)]
    assert all(torch.equal(a, b) for a, b in zip([fresh.forward(x), *fresh.backward(dy)], want))
