"""Sizes past what a launch or the kernels' 32-bit indices hold are refused as
shapes, on the host before any HIP call (no GPU needed)."""
import ctypes
import os

import pytest

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build

SHAPE = 2
P = 0x10000  # a 16-byte aligned fake address; never dereferenced on error paths


@pytest.fixture(scope="session")
def L():
    if not os.path.exists(bfp8_build.LIB_PATH):
        bfp8_build.build()
    return bfp8.lib()


def forward(L, s):
    h = bfp8.Heads(P, s.heads * s.head_dim, s.head_dim)
    return L.bfp8_attention_forward(ctypes.byref(s), h, h, h, h, P, None, 0, None)


def backward(L, s):
    h = bfp8.Heads(P, s.heads * s.head_dim, s.head_dim)
    return L.bfp8_attention_backward(ctypes.byref(s), h, h, h, h, P, h, h, h, h, P, 1 << 62, None)


def shape(total_q, total_k, heads=1, kv=1, dim=8, batch=1, causal=0):
    return bfp8.AttentionShape(batch, total_q, total_k, P, P, None, heads, kv, dim, causal, 1.0)


# A launch has fewer than 2^32 threads.
# 512 to 256 rows of a kv head:
LONG = [(1 << 29, 64, 4, 4), (1 << 30, 64, 2, 2), ((1 << 31) - 255, 1, 1, 1)]
# (in the gradient also to 128 keys)
LONG_KEYS = [(64, 1 << 30, 1, 1), (64, 1 << 28, 4, 4)]
# 16 to the statistics of a row and head:
ROWS = [(1 << 24, 64, 16, 1), (1 << 20, 64, 256, 256)]


@pytest.mark.parametrize("sizes", LONG, ids=str)
def test_long_forward(L, sizes):
    assert forward(L, shape(*sizes)) == SHAPE


@pytest.mark.parametrize("sizes", LONG + LONG_KEYS + ROWS, ids=str)
def test_long_backward(L, sizes):
    assert backward(L, shape(*sizes)) == SHAPE


@pytest.mark.parametrize("tokens,heads,dim,rot,dt", [(1 << 24, 1, 512, 510, 0), (1 << 20, 64, 256, 2, 0),
                                                     (1 << 29, 1, 128, 128, 0),
                                                     (1 << 28, 1, 128, 128, 1)])
def test_long_rope(L, tokens, heads, dim, rot, dt):
    """256 threads to as many heads as their 16-byte units (or pairs) fill."""
    for x, y in ((P, P + (1 << 40)),):
        assert L.bfp8_rope(x, heads * dim, dim, y, heads * dim, dim, dt, tokens, heads, dim, rot, 0, P,
                           100, P, 0, None) == SHAPE


def test_long_table(L):
    for n, rot in ((1 << 24, 512), (1 << 30, 8), ((1 << 31) - 1, 64)):
        assert L.bfp8_rope_table(P, n, rot, 1e4, 0, 1.0, 0, None) == SHAPE


@pytest.mark.parametrize("total_q,total_k", [(1, (1 << 31) - 1), (64, (1 << 31) - 575), (512, (1 << 31) - 513),
                                             (1 << 30, (1 << 30) - 511)])
@pytest.mark.parametrize("causal", [0, 1])
def test_rows_and_keys_together(L, total_q, total_k, causal):
    """Without a causal mask query i's last key was i + total_k in 32 bits: past
    2^31 it came out negative and the query saw nothing; and the streamed keys
    of (1, 2^31 - 1) were counted as total_k + 31."""
    s = shape(total_q, total_k, causal=causal)
    for back in (0, 1):
        assert L.bfp8_attention_workspace_bytes(ctypes.byref(s), back) == ctypes.c_size_t(-1).value
    assert forward(L, s) == SHAPE and backward(L, s) == SHAPE
