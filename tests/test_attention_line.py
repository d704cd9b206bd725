"""The line of key tiles that few query rows stream over is counted in 32 bits:
it is used only for shapes whose line fits, whatever the device arrays hold (no
GPU needed: the plan is the host's, and its workspace shows which one it is)."""
import ctypes

import pytest

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build

P = 0x10000
STREAMS = 1024  # stretches of the line


@pytest.fixture(scope="session")
def L():
    import os
    if not os.path.exists(bfp8_build.LIB_PATH):
        bfp8_build.build()
    return bfp8.lib()


def streamed(L, batch, total_q, total_k, heads, kv, dim):
    s = bfp8.AttentionShape(batch, total_q, total_k, P, P, P, heads, kv, dim, 1, 0.125)
    return L.bfp8_attention_workspace_bytes(ctypes.byref(s), 0) == 2 * STREAMS * 32 * (dim + 2) * 4


def longest_line(batch, total_q, total_k, heads, kv):
    """Every sequence has all rows and all keys, as starts that fall and rise give."""
    segments = (total_q * (heads // kv) + 31) // 32 * kv
    return batch * segments * (1 + max((total_k + 31) // 32, 1))


SHAPES = [(128, 8192, 1 << 23, 1, 1, 8), (64, 4000, 1 << 25, 2, 2, 64), (255, 255, 1 << 28, 1, 1, 8),
          (1, 8192, (1 << 31) - 1, 1, 1, 8), (2, 64, 1 << 30, 128, 1, 8), (256, 8192, 1 << 24, 1, 1, 8),
          (32, 2048, 32 << 18, 4, 1, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_streamed_lines_fit(L, shape):
    if streamed(L, *shape):
        # starts of stretches are rounded up, each by less than their number
        assert longest_line(*shape[:5]) + STREAMS < 1 << 31


# (batch, total_q, total_k, heads, kv heads, head size): requests over caches with room
SERVED = [(16, 16, 16 * 4096, 16, 8, 128), (1, 1, 131072, 16, 8, 128), (32, 32, 32 << 18, 16, 8, 128),
          (4, 20, 4 << 20, 8, 8, 64), (256, 256, 256 * 16384, 2, 1, 128)]


@pytest.mark.parametrize("shape", SERVED, ids=str)
def test_usual_caches_are_streamed(L, shape):
    assert streamed(L, *shape)
    assert longest_line(*shape[:5]) + STREAMS < 1 << 31
