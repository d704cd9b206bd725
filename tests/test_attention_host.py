"""Refusals of the attention and rotary entry points, on the host before any
HIP call (no GPU needed), and the header against the binding."""
import ctypes
import os
import re

import pytest
import torch

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bfp8_attention.h")
OK, NULL, SHAPE, ALIGN, DTYPE, LAYOUT, SMODE, WS = range(8)
P = 0x10000  # a 16-byte aligned fake address; never dereferenced on error paths
BAD = ctypes.c_size_t(-1).value


@pytest.fixture(scope="session")
def L():
    if not os.path.exists(bfp8_build.LIB_PATH):
        bfp8_build.build()
    return bfp8.lib()


def test_header_and_library_agree(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:bfp8_status|size_t)\s+(bfp8_\w+)\s*\(", src, flags=re.M))
    assert names == {"bfp8_rope_table", "bfp8_rope", "bfp8_attention_workspace_bytes",
                     "bfp8_attention_forward", "bfp8_attention_backward"}
    for name in names:
        assert hasattr(L, name)
    assert ctypes.sizeof(bfp8.AttentionShape) == 72 and ctypes.sizeof(bfp8.Heads) == 24


def shape(**k):
    d = dict(batch=2, total_q=100, total_k=200, cu_q=P, cu_k=P, k_lens=None, heads=4, kv_heads=2,
             head_dim=64, causal=1, scale=0.125)
    d.update(k)
    return bfp8.AttentionShape(*d.values())


GOOD = bfp8.Heads(P, 256, 64)
BAD_SHAPES = [dict(batch=-1), dict(total_q=-1), dict(total_k=-1), dict(heads=0), dict(kv_heads=0),
              dict(heads=5), dict(head_dim=0), dict(head_dim=12), dict(head_dim=136),
              dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(total_q=1 << 31), dict(total_k=1 << 31),
              dict(total_q=1 << 30), dict(batch=0), dict(cu_q=None, total_q=101),
              dict(cu_k=None, total_k=201)]


@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_bad_shapes(L, bad):
    s = ctypes.byref(shape(**bad))
    assert L.bfp8_attention_workspace_bytes(s, 0) == BAD
    assert L.bfp8_attention_workspace_bytes(s, 1) == BAD
    assert L.bfp8_attention_forward(s, GOOD, GOOD, GOOD, GOOD, P, None, 0, None) == SHAPE
    assert L.bfp8_attention_backward(s, GOOD, GOOD, GOOD, GOOD, P, GOOD, GOOD, GOOD, GOOD, P,
                                     1 << 30, None) == SHAPE


BAD_TENSORS = [(bfp8.Heads(None, 256, 64), NULL), (bfp8.Heads(P + 8, 256, 64), ALIGN),
               (bfp8.Heads(P, 260, 64), ALIGN), (bfp8.Heads(P, 256, 68), ALIGN),
               (bfp8.Heads(P, 56, 64), SHAPE), (bfp8.Heads(P, 256, 56), SHAPE),
               (bfp8.Heads(P, (1 << 22) + 8, 64), SHAPE), (bfp8.Heads(P, 256, -64), SHAPE)]


@pytest.mark.parametrize("bad,status", BAD_TENSORS)
def test_bad_tensors(L, bad, status):
    s = ctypes.byref(shape())
    for i in range(4):
        t = [GOOD] * 4
        t[i] = bad
        assert L.bfp8_attention_forward(s, *t, P, None, 0, None) == status
    for i in range(8):
        t = [GOOD] * 8
        t[i] = bad
        assert L.bfp8_attention_backward(s, *t[:4], P, *t[4:], P, 1 << 30, None) == status


def test_other_pointers_and_workspace(L):
    s = ctypes.byref(shape())
    F = lambda lse=P, ws=None, n=0: L.bfp8_attention_forward(s, GOOD, GOOD, GOOD, GOOD, lse, ws, n,
                                                             None)
    assert F(lse=None) == NULL and F(lse=P + 4) == ALIGN and F(ws=P + 4, n=100) == ALIGN
    B = lambda lse=P, ws=P, n=1 << 30: L.bfp8_attention_backward(
        s, GOOD, GOOD, GOOD, GOOD, lse, GOOD, GOOD, GOOD, GOOD, ws, n, None)
    assert B(lse=None) == NULL and B(lse=P + 4) == ALIGN and B(ws=P + 4) == ALIGN
    need = L.bfp8_attention_workspace_bytes(s, 1)
    assert 0 < need < 1 << 20
    assert B(ws=None) == WS and B(n=need - 1) == WS
    assert L.bfp8_attention_forward(None, GOOD, GOOD, GOOD, GOOD, P, None, 0, None) == NULL
    assert L.bfp8_attention_workspace_bytes(s, 2) == BAD


def test_empty_problems_need_nothing(L):
    N = bfp8.Heads(None, 0, 0)
    for kw in (dict(batch=0, total_q=0, total_k=0, cu_q=None, cu_k=None),
               dict(total_q=0, total_k=0, cu_q=None, cu_k=None)):
        s = ctypes.byref(shape(**kw))
        assert L.bfp8_attention_forward(s, N, N, N, N, None, None, 0, None) == OK
        assert L.bfp8_attention_backward(s, N, N, N, N, None, N, N, N, N, None, 0, None) == OK


def rope(L, x=P, xr=256, xh=64, y=P + 4096, yr=256, yh=64, dt=0, T=10, H=4, D=64, rot=64, layout=0,
         table=P, rows=100, pos=P, inverse=0):
    return L.bfp8_rope(x, xr, xh, y, yr, yh, dt, T, H, D, rot, layout, table, rows, pos, inverse,
                       None)


def test_rope_refusals(L):
    assert rope(L, dt=2) == DTYPE
    assert rope(L, layout=2) == LAYOUT
    assert rope(L, x=None) == NULL and rope(L, y=None) == NULL and rope(L, table=None) == NULL
    assert rope(L, x=P + 8) == ALIGN and rope(L, y=P + 2) == ALIGN and rope(L, table=P + 4) == ALIGN
    assert rope(L, xr=260) == ALIGN and rope(L, yh=68) == ALIGN
    for bad in (dict(T=-1), dict(H=-1), dict(D=0), dict(D=60), dict(D=520), dict(rot=0),
                dict(rot=66), dict(rot=63), dict(inverse=2), dict(rows=0), dict(rows=-1),
                dict(xr=56), dict(yh=56), dict(x=P, y=P, yr=512), dict(T=1 << 30)):
        assert rope(L, **bad) == SHAPE, bad
    assert rope(L, T=0, x=None, y=None, table=None) == OK
    assert rope(L, H=0, x=None, y=None, table=None) == OK


def test_rope_table_refusals(L):
    T = lambda table=P, n=100, rot=64, base=1e4, scaling=0, factor=1.0, original=0: \
        L.bfp8_rope_table(table, n, rot, base, scaling, factor, original, None)
    assert T(scaling=4) == LAYOUT and T(scaling=-1) == LAYOUT
    for bad in (dict(n=-1), dict(rot=0), dict(rot=63), dict(rot=514), dict(base=0.0),
                dict(base=float("nan")), dict(scaling=1, factor=0.5),
                dict(scaling=2, factor=float("inf")), dict(scaling=3, factor=2.0), dict(n=1 << 31)):
        assert T(**bad) == SHAPE, bad
    assert T(table=None) == NULL and T(table=P + 4) == ALIGN
    assert T(table=None, n=0) == OK


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        bfp8.attention_forward(x, x, x)
    with pytest.raises(ValueError, match="device tensor"):
        bfp8.rope(x, torch.zeros((4, 32, 2)))
    with pytest.raises(ValueError, match="scaling"):
        bfp8.rope_table(4, 64, scaling="dynamic")
    with pytest.raises(ValueError, match="layout"):
        bfp8.rope(x, torch.zeros((4, 32, 2)), layout="pairs")
