"""What the binding passes on for one token of a tensor stored head by head
(no GPU needed: the strides are checked on the host before any HIP call)."""
import torch

from blockwise_fp8_gemm_bfp8_amd import attention

MAX_ROW = 1 << 22  # the library's largest row stride, in elements


class OnDevice:
    """The sizes and strides of a tensor, said to be on device 0."""

    def __init__(self, t):
        self.shape, self.dtype, self.stride, self.data_ptr = t.shape, t.dtype, t.stride, t.data_ptr
        self.get_device = lambda: 0


def test_one_token_of_head_major_tensors():
    room = torch.empty((8, 8192, 128), dtype=torch.bfloat16, device="meta").transpose(0, 1)
    for n in (1, 2):
        _, size, h = attention._heads(OnDevice(room[5:5 + n]), "k", (torch.bfloat16,))
        assert tuple(size) == (n, 8, 128) and h.head == 1 << 20
        assert 128 <= h.row <= MAX_ROW and h.row % 8 == 0
