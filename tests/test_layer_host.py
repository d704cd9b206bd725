"""The layer operators' refusals and host logic, without a GPU: every status
comes before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd import build as bfp8_build
from blockwise_fp8_gemm_bfp8_amd.mlp_block import MLPBlock

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, DTYPE, LAYOUT, SMODE, WS = range(8)
P = 0x10000  # an aligned fake address; never dereferenced on error paths
BF, F32 = 0, 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bfp8_build.LIB_PATH):
        bfp8_build.build()
    return bfp8.lib()


def test_header_and_exports(L):
    src = open(os.path.join(ROOT, "include", "bfp8_layer.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:bfp8_status|size_t)\s+(bfp8_\w+)\s*\(", src, flags=re.M))
    assert names == {"bfp8_rmsnorm", "bfp8_rmsnorm_quantize", "bfp8_rmsnorm_backward",
                     "bfp8_rmsnorm_backward_workspace_bytes", "bfp8_swiglu", "bfp8_swiglu_quantize",
                     "bfp8_swiglu_backward", "bfp8_swiglu_backward_quantize", "bfp8_grad_norm",
                     "bfp8_grad_norm_workspace_bytes", "bfp8_grad_clip", "bfp8_grad_norm_clip"}
    for name in names:
        assert hasattr(L, name), name
    assert ctypes.sizeof(bfp8.GradJob) == 56


def norm(L, quantize=False, **k):
    d = dict(x=P, ldx=256, residual=None, ldres=0, w=P, wdt=F32, dt=BF, rows=128, cols=256, eps=1e-6,
             sum=None, ldsum=0)
    t = dict(rstd=P, format=0, q=P, ldq=256, s=P, qt=P, ldqt=128, st=P) if quantize else \
        dict(y=P, ldy=256, rstd=P)
    assert not set(k) - set(d) - set(t)
    fn = L.bfp8_rmsnorm_quantize if quantize else L.bfp8_rmsnorm
    return fn(*{**d, **{n: v for n, v in k.items() if n in d}}.values(),
              *{**t, **{n: v for n, v in k.items() if n in t}}.values(), None)


@pytest.mark.parametrize("quantize", [False, True])
def test_norm_refusals(L, quantize):
    call = lambda **k: norm(L, quantize, **k)
    for name in ("x", "w", "rstd"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: P + 4}) == ALIGN, name
    assert call(residual=P, ldres=256) == NULL  # no place for the sum
    assert call(residual=P, ldres=256, sum=P, ldsum=255) == SHAPE
    assert call(residual=P + 8, ldres=256, sum=P, ldsum=256) == ALIGN
    assert call(ldx=255) == SHAPE and call(ldx=257) == ALIGN and call(ldx=1 << 41) == SHAPE
    assert call(dt=2) == DTYPE and call(wdt=7) == DTYPE
    assert call(rows=-1) == SHAPE and call(cols=-1) == SHAPE and call(rows=1 << 31) == SHAPE
    assert call(cols=16512, ldx=16512) == SHAPE
    for eps in (0.0, -1.0, NAN, INF, 2.0 ** -127, 2.0 ** -149):
        assert call(eps=eps) == SHAPE, eps
    assert call(eps=2.0 ** -126, rows=0) == OK
    assert call(rows=0, x=None, w=None, rstd=None) == OK
    # rows that no 32-bit count of their vectors holds
    assert call(rows=(1 << 31) - 128, cols=256) == SHAPE
    # a result over an input whose rows lie elsewhere
    Q = P + 0x10000
    assert call(residual=Q, ldres=256, sum=Q, ldsum=264) == SHAPE
    assert call(residual=Q, ldres=256, sum=P, ldsum=264) == SHAPE
    if not quantize:
        assert call(ldy=264) == SHAPE and call(residual=Q, ldres=256, sum=P, ldsum=256) == SHAPE


def codes_refusals(call, cols):
    assert call(format=3) == SMODE and call(format=-1) == SMODE
    for name in ("q", "s", "st"):
        assert call(**{name: None}) == NULL, name
    for name in ("q", "s", "qt", "st"):
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(ldq=cols - 16) == SHAPE and call(ldqt=64) == SHAPE
    assert call(ldq=cols + 8) == ALIGN and call(ldqt=136) == ALIGN
    assert call(rows=100) == SHAPE  # token groups of 128


def test_codes_refusals(L):
    codes_refusals(lambda **k: norm(L, True, **k), 256)
    assert norm(L, True, cols=200) == SHAPE
    for grad in (False, True):
        codes_refusals(lambda **k: glu(L, grad, True, **k), 512 if grad else 256)
        assert glu(L, grad, True, cols=192) == SHAPE
    assert glu(L, False, True, rows=100, qt=None, st=None, gate=None) == NULL  # rows of any number


def glu(L, grad, quantize, **k):
    d = dict(dh=P, lddh=256) if grad else {}
    d.update(gate=P, ldg=256, up=P, ldu=256, dt=BF, rows=128, cols=256)
    if quantize:
        d.update(format=0, q=P, ldq=512 if grad else 256, s=P, qt=P, ldqt=128, st=P)
    elif grad:
        d.update(dgate=P, lddg=256, dup=P, lddu=256)
    else:
        d.update(h=P, ldh=256)
    assert not set(k) - set(d)
    name = "bfp8_swiglu" + ("_backward" if grad else "") + ("_quantize" if quantize else "")
    return getattr(L, name)(*{**d, **k}.values(), None)


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("grad", [False, True])
def test_glu_refusals(L, grad, quantize):
    call = lambda **k: glu(L, grad, quantize, **k)
    tensors = [("gate", "ldg"), ("up", "ldu")] + ([("dh", "lddh")] if grad else [])
    if not quantize:
        tensors += [("dgate", "lddg"), ("dup", "lddu")] if grad else [("h", "ldh")]
    for name, ld in tensors:
        assert call(**{name: None}) == NULL and call(**{name: P + 2}) == ALIGN, name
        assert call(**{ld: 248}) == SHAPE and call(**{ld: 260}) == ALIGN, ld
    if not quantize:  # two results in one place, or over an input whose rows lie elsewhere
        Q = P + 0x10000
        assert call(ldg=264) == SHAPE and call(ldu=264) == SHAPE
        if grad:
            assert call() == SHAPE and call(dup=Q, lddh=264) == SHAPE and call(dup=Q, ldg=264) == SHAPE
    assert call(dt=9) == DTYPE and call(rows=-1) == SHAPE and call(cols=-1) == SHAPE
    assert call(rows=1 << 31) == SHAPE and call(rows=(1 << 31) - 128) == SHAPE
    assert call(rows=0, gate=None, up=None) == OK


def test_norm_gradient_refusals(L):
    d = dict(dy=P, lddy=256, r=P, ldr=256, w=P, wdt=F32, rstd=P, dsum=P, lddsum=256, dt=BF, rows=128,
             cols=256, dx=P, lddx=256, dw=P, ws=P, nbytes=1 << 30)
    call = lambda **k: L.bfp8_rmsnorm_backward(*{**d, **k}.values(), None)
    for name in ("dy", "r", "w", "rstd", "dx", "dw"):
        assert call(**{name: None}) == NULL and call(**{name: P + 4}) == ALIGN, name
    assert call(dsum=P + 4) == ALIGN and call(ws=P + 4) == ALIGN
    for ld in ("lddy", "ldr", "lddsum", "lddx"):
        assert call(**{ld: 248}) == SHAPE and call(**{ld: 260}) == ALIGN, ld
    for ld in ("lddy", "ldr", "lddsum"):  # dx over an input whose rows lie elsewhere
        assert call(**{ld: 264}) == SHAPE
    need = L.bfp8_rmsnorm_backward_workspace_bytes(128, 256)
    assert need > 0 and need % (256 * 4) == 0
    assert call(ws=None) == WS and call(nbytes=need - 1) == WS
    assert call(dt=2) == DTYPE and call(wdt=2) == DTYPE
    assert call(rows=-1) == SHAPE and call(cols=16385) == SHAPE and call(cols=0) == OK
    assert call(rows=0, dw=None) == NULL
    assert L.bfp8_rmsnorm_backward_workspace_bytes(-1, 4) == ctypes.c_size_t(-1).value
    assert L.bfp8_rmsnorm_backward_workspace_bytes(0, 4) == 0


def test_clip_refusals(L):
    job = lambda **k: bfp8.GradJob(**{**dict(g=P, out=P, rows=4, cols=100, ldg=100, ldo=100, dt=F32), **k})

    def both(*jobs, max_norm=1.0, norm=P):
        arr = (bfp8.GradJob * max(len(jobs), 1))(*jobs)
        a = L.bfp8_grad_norm(arr, len(jobs), norm, P, 1 << 30, None)
        b = L.bfp8_grad_clip(arr, len(jobs), norm, max_norm, None)
        c = L.bfp8_grad_norm_clip(arr, len(jobs), norm, max_norm, P, 1 << 30, None)
        assert a == b == c
        return a
    assert both(job(g=None)) == NULL and both(job(), job(g=None)) == NULL
    assert both(job(g=P + 2)) == ALIGN and both(job(g=P + 1, out=P + 1, dt=BF)) == ALIGN
    assert both(job(dt=2)) == DTYPE and both(job(ldg=99, ldo=99)) == SHAPE
    assert both(job(rows=-1)) == SHAPE and both(job(cols=-1)) == SHAPE
    assert both(job(rows=1 << 20, cols=1 << 20, ldg=1 << 20, ldo=1 << 20)) == SHAPE
    assert both(job(), norm=None) == NULL and both(job(), norm=P + 2) == ALIGN
    one = (bfp8.GradJob * 1)(job())

    def clip(j, m=1.0):
        a = L.bfp8_grad_clip((bfp8.GradJob * 1)(j), 1, P, m, None)
        assert a == L.bfp8_grad_norm_clip((bfp8.GradJob * 1)(j), 1, P, m, P, 1 << 30, None)
        return a
    assert clip(job(out=None)) == NULL and clip(job(out=P + 2)) == ALIGN and clip(job(ldo=99)) == SHAPE
    assert clip(job(ldo=128)) == SHAPE  # in place, with another row stride
    assert clip(job(), -1.0) == SHAPE and clip(job(), NAN) == SHAPE
    assert L.bfp8_grad_norm(one, -1, P, P, 1 << 30, None) == SHAPE
    assert L.bfp8_grad_norm(None, 1, P, P, 1 << 30, None) == NULL
    assert L.bfp8_grad_clip(None, 0, None, 1.0, None) == OK
    need = L.bfp8_grad_norm_workspace_bytes(one, 1)
    assert need == 8 and L.bfp8_grad_norm(one, 1, P, P, 7, None) == WS
    assert L.bfp8_grad_norm(one, 1, P, None, 8, None) == WS
    assert L.bfp8_grad_norm(one, 1, P, P + 8, 8, None) == ALIGN
    assert L.bfp8_grad_norm_clip(one, 1, P, 1.0, P, 7, None) == WS
    empty = (bfp8.GradJob * 1)(job(g=None, out=None, cols=0))
    assert L.bfp8_grad_norm_workspace_bytes(empty, 1) == 0 and L.bfp8_grad_clip(empty, 1, P, 1.0, None) == OK
    assert L.bfp8_grad_norm_workspace_bytes(one, -1) == ctypes.c_size_t(-1).value
    # many tensors are several launches with sums of their own
    many = (bfp8.GradJob * 165)(*[job()] * 165)
    assert L.bfp8_grad_norm_workspace_bytes(many, 165) == 165 * 8


def test_binding_refuses_host_tensors():
    x, w = torch.zeros((4, 128)), torch.ones(128)
    for call in (lambda: bfp8.rmsnorm(x, w), lambda: bfp8.rmsnorm_quantize(x, w),
                 lambda: bfp8.rmsnorm_backward(x, x, w, torch.ones(4)), lambda: bfp8.swiglu(x, x),
                 lambda: bfp8.swiglu_quantize(x, x), lambda: bfp8.swiglu_backward(x, x, x),
                 lambda: bfp8.GradClip([x]), lambda: bfp8.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError):
        bfp8.GradClip([])


def test_mlp_block_sizes():
    bf = torch.bfloat16
    w = lambda *s: torch.zeros(s, dtype=bf)
    with pytest.raises(ValueError, match="w_gate_up"):
        MLPBlock(w(128), w(256, 128), w(128, 256), 128)
    with pytest.raises(ValueError, match="w_norm"):
        MLPBlock(w(256), w(512, 128), w(128, 256), 128)
    for hidden, ffn, tokens in ((128, 256, 100), (130, 256, 128), (128, 200, 128)):
        with pytest.raises(ValueError, match="multiple of 128"):
            MLPBlock(w(hidden), w(2 * ffn, hidden), w(hidden, ffn), tokens)
