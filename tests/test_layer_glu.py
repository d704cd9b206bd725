"""The gated activation, its gradient and the codes of both against float64.

With U = 2^-24: the exponent's argument is |g| log2(e) within 1.5 U of itself, so
exp(-g) is within (1.5 |g| + 2) U; the addition, the reciprocal (one step: 2 U)
and the products add 8 U at most, so sigma and silu are within (1.5 |g| + 12) U.
For |g| > 87 sigma is held at 2^-126: |g| up 2^-125 is added.  In dgate's factor
1 + g (1 - sigma) both terms' sizes count."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import U, as_quantised, check_codes, close, f64, generator, padded  # noqa: E402
from oracle import layer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (3, 8), (37, 100), (5, 129), (130, 2047), (2, 6144), (1, 20001)]


def inputs(rows, cols, dtype, seed, extra=0):
    gen = generator(seed)
    gate, up = padded(rows, cols, dtype, gen, 3.0, extra), padded(rows, cols, dtype, gen, 1.5, 2 * extra)
    if rows * cols > 64:  # where the exponential is huge, tiny, or leaves float32
        flat = torch.tensor([30.0, -30.0, 90.0, -90.0, 200.0, -200.0, 0.0, -1.278], device="cuda").to(dtype)
        gate[0, :8] = flat
    return gate, up, padded(rows, cols, dtype, gen, 1e-3, extra)


def reach(gate, up):
    """Errors of h, and of dgate and dup for dh = 1."""
    g, u = np.abs(f64(gate)), np.abs(f64(up))
    sig = layer._sigma(f64(gate))
    rel = (3 * g + 24) * U
    floor = (1 + g) * 2.0 ** -125
    return (rel * g * sig * u + floor * u, u * (rel * sig * (1 + g * (1 - sig)) + floor),
            rel * g * sig + floor)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_values_and_gradient(rows, cols, dtype):
    gate, up, dh = inputs(rows, cols, dtype, cols, rows % 3)
    e, eg, eu = reach(gate, up)
    close(bfp8.swiglu(gate, up), layer.swiglu(f64(gate), f64(up)), e, dtype)
    dgate, dup = bfp8.swiglu_backward(dh, gate, up)
    wg, wu = layer.swiglu_backward(f64(dh), f64(gate), f64(up))
    size = np.abs(f64(dh))
    close(dgate, wg, eg * size, dtype)
    close(dup, wu, eu * size, dtype)


@pytest.mark.parametrize("scales", ["fp32", "mx128", "mx32"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,transposed", [(1, 128, False), (7, 640, False), (33, 6144, False),
                                                  (128, 128, True), (384, 640, True), (128, 6144, True)])
def test_codes(rows, cols, transposed, dtype, scales):
    gate, up, dh = inputs(rows, cols, dtype, rows + cols, 1)
    e, eg, eu = reach(gate, up)
    out = bfp8.swiglu_quantize(gate, up, scales=scales, transposed=transposed)
    check_codes(out, layer.swiglu(f64(gate), f64(up)), e, scales)
    y32 = bfp8.swiglu(gate.float(), up.float())
    for a, b in zip(out, as_quantised(bfp8, y32, scales, transposed)):
        assert torch.equal(a, b)
    out = bfp8.swiglu_backward_quantize(dh, gate, up, scales=scales, transposed=transposed)
    size = np.abs(f64(dh))
    check_codes(out, np.concatenate(layer.swiglu_backward(f64(dh), f64(gate), f64(up)), 1),
                np.concatenate([eg * size, eu * size], 1), scales)
    y32 = torch.cat(bfp8.swiglu_backward(dh.float(), gate.float(), up.float()), 1)
    for a, b in zip(out, as_quantised(bfp8, y32, scales, transposed)):
        assert torch.equal(a, b)


def test_halves_of_one_projection_and_in_place():
    gate_up = torch.randn((50, 512), device="cuda", generator=generator(1)).to(BF)
    gate, up = gate_up[:, :256], gate_up[:, 256:]
    dh = torch.randn((50, 256), device="cuda", generator=generator(2)).to(BF)
    dgate, dup = bfp8.swiglu_backward(dh, gate.contiguous(), up.contiguous())
    h = bfp8.swiglu(gate.contiguous(), up.contiguous())
    rows = gate_up.clone()
    bfp8.swiglu(rows[:, :256], rows[:, 256:], out=rows[:, :256])
    assert torch.equal(rows[:, :256], h) and torch.equal(rows[:, 256:], up)
    rows = gate_up.clone()  # the gradient over its own inputs
    bfp8.swiglu_backward(dh, rows[:, :256], rows[:, 256:], dgate=rows[:, :256], dup=rows[:, 256:])
    assert torch.equal(rows[:, :256], dgate) and torch.equal(rows[:, 256:], dup)


@pytest.mark.parametrize("scales", ["fp32", "mx128", "mx32"])
def test_groups_of_tiny_and_zero_results(scales):
    """Gates far below zero make whole groups of results that no float32 scale
    covers: they count as zeros, in both layouts, and their neighbours are as ever."""
    gate = torch.randn((256, 256), device="cuda", generator=generator(3))
    up = torch.randn((256, 256), device="cuda", generator=generator(4))
    gate[5, :128] = -100.0   # a row group
    gate[128:, 200] = -95.0  # a token group
    up[7] = 0.0
    q, s, qt, st = bfp8.swiglu_quantize(gate, up, scales=scales, transposed=True)
    assert not torch.any((q & 0x7F) == 0x7F) and not torch.any((qt & 0x7F) == 0x7F)
    assert torch.all(q[7] & 0x7F == 0)
    e, _, _ = reach(gate, up)
    check_codes((q, s, qt, st), layer.swiglu(f64(gate), f64(up)), e, scales)
    if scales == "fp32":
        assert s[0, 5] == 1 and torch.all(q[5, :128] & 0x7F == 0)
        assert st[1, 200] == 1 and torch.all(qt[200, 128:] & 0x7F == 0)


def test_nan_stays_in_its_groups():
    gate = torch.randn((128, 384), device="cuda", generator=generator(5))
    up = torch.randn((128, 384), device="cuda", generator=generator(6))
    clean = bfp8.swiglu_quantize(gate, up, transposed=True)
    gate[3, 130] = float("nan")
    up[9, 131] = float("inf")
    q, s, qt, st = bfp8.swiglu_quantize(gate, up, transposed=True)
    rows = torch.ones((128, 384), dtype=torch.bool, device="cuda")
    rows[3, 128:256] = rows[9, 128:256] = False
    assert torch.equal(q[rows], clean[0][rows])
    cols = torch.ones(384, dtype=torch.bool, device="cuda")
    cols[130:132] = False
    assert torch.equal(qt[cols], clean[2][cols]) and torch.equal(st[:, cols], clean[3][:, cols])


def test_empty():
    none = torch.empty((0, 128), dtype=BF, device="cuda")
    assert bfp8.swiglu(none, none).shape == (0, 128)
    q, s, qt, st = bfp8.swiglu_backward_quantize(none, none, none, transposed=True)
    assert q.shape == (0, 256) and s.shape == (2, 0) and qt.shape == (256, 0) and st.shape == (0, 256)
