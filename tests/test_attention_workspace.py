"""A workspace that is given must be memory the kernels can use: dense, on the
device of the call."""
import pytest
import torch

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd import attention


class OnDevice:
    def get_device(self):
        return 0


@pytest.mark.parametrize("backward", [0, 1])
def test_host_memory_is_refused(backward):
    """Without a GPU: the check comes before any HIP call."""
    shape = bfp8.AttentionShape(1, 64, 64, None, None, None, 1, 1, 64, 1, 0.125)
    with pytest.raises(ValueError, match="workspace"):
        attention._workspace(shape, backward, torch.empty(1 << 20, dtype=torch.uint8), OnDevice())


@pytest.mark.gpu
def test_given_workspaces():
    gen = torch.Generator(device="cuda").manual_seed(51)
    new = lambda h: torch.randn((2000, h, 64), device="cuda", generator=gen).to(torch.bfloat16)
    q, k, v, do = new(2), new(1), new(1), new(2)
    o, lse = bfp8.attention_forward(q, k, v)
    want = bfp8.attention_backward(do, q, k, v, o, lse)
    need = [bfp8.attention_workspace_bytes(q, k, v, backward=back) for back in (False, True)]
    assert min(need) > 0
    n = (max(need) // 16 + 1) * 4
    room = torch.empty(2 * n, dtype=torch.float32, device="cuda")
    bad = [torch.empty(n), torch.empty(1, device="cuda").expand(n), room[::2],
           room.view(n, 2)[:, 0], room.view(2, n).t()]
    for ws in bad:
        with pytest.raises(ValueError, match="workspace"):
            bfp8.attention_forward(q, k, v, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            bfp8.attention_backward(do, q, k, v, o, lse, workspace=ws)
    for ws in (room[:n], room[n:].view(torch.uint8), room[:n].view(1, n)):
        o2, lse2 = bfp8.attention_forward(q, k, v, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        got = bfp8.attention_backward(do, q, k, v, o, lse, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
