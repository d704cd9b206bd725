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
