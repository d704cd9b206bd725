"""RMS norm, its codes and its gradient against float64 (oracle/layer.py).

Tolerances count float32 roundings (U = 2^-24 relative each).  A row's sum of
squares is a chain of at most 32 and a tree of at most 10 additions, halved by
the root; the mean, eps, the root, the reciprocal and two products add 7 at
most: y is within 28 U of exact; NORM takes 32.  The gradient's terms g and t mean are each
within 3 U + (the mean's error, that of a sum of 42 additions of its terms'
sizes), times rstd."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import EPS, HALF, U, as_quantised, check_codes, close, f64, generator, padded  # noqa: E402
from oracle import layer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NORM = 32 * U
# every number of threads and vectors a row takes, with tails and single columns
SIZES = [(1, 1), (3, 8), (37, 100), (16, 128), (5, 129), (9, 511), (6, 1000), (7, 2048), (130, 2047),
         (3, 2049), (2, 4096), (2, 5000), (1, 8192), (3, 8200), (2, 16384), (1, 12345)]


def inputs(rows, cols, dtype, seed, added, wdt=F32, extra=0):
    gen = generator(seed)
    x = padded(rows, cols, dtype, gen, 2.0, extra)
    residual = padded(rows, cols, dtype, gen, 1.0, 2 * extra) if added else None
    w = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)).to(wdt)
    stored = x if residual is None else (x.float() + residual.float()).to(dtype)
    return x, residual, w, stored


@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_values(rows, cols, dtype, added):
    x, residual, w, stored = inputs(rows, cols, dtype, cols, added, BF if rows % 2 else F32, rows % 3)
    y, r, rstd = bfp8.rmsnorm(x, w, residual, eps=EPS)
    assert torch.equal(r, stored) and (r is x) == (not added)
    want, stat = layer.rmsnorm(f64(stored), f64(w), EPS)
    close(rstd, stat, NORM * stat)
    close(y, want, NORM * np.abs(want), dtype)


def test_padding_and_inputs_stay():
    x, residual, w, _ = inputs(5, 100, BF, 1, True, extra=2)
    out, total = padded(5, 100, BF, generator(2), extra=1), padded(5, 100, BF, generator(3), extra=1)
    before = x.clone(), residual.clone()
    bfp8.rmsnorm(x, w, residual, out=out, sum_out=total)
    assert torch.equal(x, before[0]) and torch.equal(residual, before[1])
    for t in (out, total):
        assert torch.all(t._base[:, 100:] == 777)


def test_in_place():
    x, residual, w, stored = inputs(70, 1000, BF, 4, True)
    y, r, rstd = bfp8.rmsnorm(x, w, residual)
    a, b = x.clone(), residual.clone()
    y2, r2, rstd2 = bfp8.rmsnorm(a, w, b, out=a, sum_out=b)  # both inputs given up
    assert r2 is b and torch.equal(y, y2) and torch.equal(r, r2) and torch.equal(rstd, rstd2)
    c = x.clone()
    assert torch.equal(bfp8.rmsnorm(c, w, out=c)[0], bfp8.rmsnorm(x, w)[0])


def test_rows_of_zeros_and_one_value():
    x = torch.zeros((3, 256), dtype=BF, device="cuda")
    x[1, 7] = 3.0
    w = torch.ones(256, device="cuda")
    y, _, rstd = bfp8.rmsnorm(x, w, eps=EPS)
    assert torch.all(y[0] == 0) and torch.all(y[2] == 0)
    assert torch.count_nonzero(y[1]) == 1
    close(y[1, 7:8], np.array([16.0 * (1 + EPS * 256 / 9) ** -0.5]), 32 * NORM, BF)
    q, s, _, _ = bfp8.rmsnorm_quantize(x, w, eps=EPS)
    assert torch.all(q[0] == 0) and torch.all(s[:, 0] == 1) and torch.all(s[1] == 1)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e30])
def test_smallest_and_large_eps(eps):
    """Rows of zeros under the smallest eps, whose root is 2^63, and rows whose squares
    vanish beside it or outweigh it."""
    x = torch.zeros((4, 300), device="cuda")
    x[1:] = torch.randn((3, 300), device="cuda", generator=generator(8))
    x[2] *= 1e-17
    x[3] *= 1e15
    w = torch.ones(300, device="cuda")
    y, r, rstd = bfp8.rmsnorm(x, w, eps=eps)
    want, stat = layer.rmsnorm(f64(x), f64(w), eps)
    close(rstd, stat, NORM * stat)
    close(y, want, NORM * np.abs(want) + 2.0 ** -126)  # results below that may vanish
    assert torch.all(y[0] == 0)


@pytest.mark.parametrize("scales", ["fp32", "mx128", "mx32"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,transposed", [(1, 128, False), (7, 512, False), (33, 2048, False),
                                                  (3, 4224, False), (2, 9088, False), (1, 16384, False),
                                                  (128, 128, True), (384, 640, True), (128, 4352, True),
                                                  (256, 16384, True)])
def test_codes(rows, cols, transposed, dtype, scales):
    x, residual, w, stored = inputs(rows, cols, dtype, rows, rows % 2 == 0, BF if cols > 600 else F32, 1)
    *out, r, rstd = bfp8.rmsnorm_quantize(x, w, residual, eps=EPS, scales=scales, transposed=transposed)
    assert torch.equal(r, stored) and len(out) == (4 if transposed else 2)
    want, stat = layer.rmsnorm(f64(stored), f64(w), EPS)
    close(rstd, stat, NORM * stat)
    check_codes(out, want, NORM * np.abs(want), scales)
    # the same bytes as the quantisers' on the float32 result
    y32, _, _ = bfp8.rmsnorm(stored.float(), w, eps=EPS)
    for a, b in zip(out, as_quantised(bfp8, y32, scales, transposed)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES + [(5000, 64), (4101, 300), (2100, 4100)])
def test_gradient(rows, cols, dtype, added):
    x, dsum, w, _ = inputs(rows, cols, dtype, cols + rows, added, BF if rows % 2 else F32, rows % 3)
    dy = padded(rows, cols, dtype, generator(5), 1e-3, rows % 2)
    _, r, rstd = bfp8.rmsnorm(x, w, eps=EPS)
    dx, dw = bfp8.rmsnorm_backward(dy, r, w, rstd, dsum)
    a, b, c = f64(dy), f64(r), f64(w)
    want_dx, want_dw = layer.rmsnorm_backward(a, b, c, EPS, f64(dsum) if added else None)
    _, s = layer.rmsnorm(b, c, EPS)
    t, g = np.abs(b * s[:, None]), np.abs(a * c)
    # sizes of the terms, each within 64 U with rstd's own error
    err = 64 * U * s[:, None] * (g + t * np.mean(g * t, axis=1)[:, None])
    if added:
        err = err + U * np.abs(f64(dsum))
    close(dx, want_dx, err, dtype)
    # a column's sum: each row's term within 40 U, at most 100 additions on its way
    close(dw, want_dw, 140 * U * np.sum(np.abs(a) * t, axis=0))


def test_gradient_against_differences():
    """The calls alone: (L(r + h d) - L(r - h d)) / 2h for L = sum(dy y).  float32
    values of y have errors of NORM each, over 2h; the second-order term is h^2."""
    gen = generator(8)
    rows, cols, h = 4, 192, 1e-2
    r, dy, d = (torch.randn((rows, cols), device="cuda", generator=gen) for _ in range(3))
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
    _, _, rstd = bfp8.rmsnorm(r, w)
    dx, dw = bfp8.rmsnorm_backward(dy, r, w, rstd)
    up, down = (bfp8.rmsnorm((r.double() + s * h * d.double()).float(), w)[0].double() for s in (1, -1))
    got = ((up - down) * dy).sum().item() / (2 * h)
    noise = 2 * NORM * (up.abs() * dy.abs()).sum().item() / (2 * h)
    third = 20 * h * h * (dy.abs() * d.abs()).sum().item()  # derivatives of a unit-scale row are O(1)
    assert abs(got - (dx * d).sum().item()) <= noise + third
    e = torch.randn(cols, device="cuda", generator=gen)
    up, down = (bfp8.rmsnorm(r, w + s * e)[0].double() for s in (1, -1))  # linear in w
    assert abs(((up - down) * dy).sum().item() / 2 - (dw * e).sum().item()) <= \
        200 * U * (dy.abs() * r.abs() * rstd[:, None] * (w.abs() + e.abs())).sum().item()


def test_gradient_in_place_and_over_no_rows():
    x, dsum, w, _ = inputs(300, 700, BF, 9, True)
    dy = padded(300, 700, BF, generator(10), 1e-3)
    _, r, rstd = bfp8.rmsnorm(x, w)
    dx, dw = bfp8.rmsnorm_backward(dy, r, w, rstd, dsum)
    for give in range(3):
        a, b, c = (t._base.clone()[:, :700] for t in (dy, r, dsum))  # rows stay 16-byte aligned
        dx2, dw2 = bfp8.rmsnorm_backward(a, b, w, rstd, c, dx=(a, b, c)[give])
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    none = torch.empty((0, 700), dtype=BF, device="cuda")
    dx, dw = bfp8.rmsnorm_backward(none, none, w, torch.empty(0, device="cuda"),
                                   dweight=torch.full((700,), 5.0, device="cuda"))
    assert dx.shape == (0, 700) and torch.all(dw == 0)


def test_offsets_past_32_bits():
    """Rows so far apart that the last starts past 2^32 elements."""
    rows, cols, ld = 140, 256, 1 << 25
    base = torch.empty(rows * ld, dtype=BF, device="cuda")
    x = base.view(rows, ld)[:, :cols]
    x.copy_(torch.randn((rows, cols), device="cuda", generator=generator(11)))
    w = torch.ones(cols, device="cuda")
    dense = x.contiguous()
    y, _, rstd = bfp8.rmsnorm(dense, w)
    out = base.view(rows, ld)[:, cols:2 * cols]
    assert torch.equal(bfp8.rmsnorm(x, w, out=out)[0], y) and torch.equal(out, y)
    top = x[:128]
    for a, b in zip(bfp8.rmsnorm_quantize(top, w, transposed=True),
                    bfp8.rmsnorm_quantize(dense[:128], w, transposed=True)):
        assert torch.equal(a, b)
    dx, dw = bfp8.rmsnorm_backward(out, x, w, rstd)
    dx2, dw2 = bfp8.rmsnorm_backward(y, dense, w, rstd)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    gate, up = x, base.view(rows, ld)[:, 2 * cols:3 * cols]
    up.copy_(dense * 0.5)
    assert torch.equal(bfp8.swiglu(gate, up), bfp8.swiglu(dense, dense * 0.5))


def test_many_rows_of_few_channels():
    """The norm of heads: more rows than workgroups start at once."""
    rows = (1 << 21) + 5
    x = torch.randn((rows, 64), device="cuda", generator=generator(12)).to(BF)
    w = torch.ones(64, device="cuda")
    y, _, _ = bfp8.rmsnorm(x, w)
    for at in (slice(0, 300), slice(1 << 20, (1 << 20) + 300), slice(rows - 300, rows)):
        assert torch.equal(y[at], bfp8.rmsnorm(x[at], w)[0])


def test_more_rows_than_workgroups():
    """Rows of several waves, in turn: each turn's sums are its own."""
    rows = (1 << 16) + 4000
    x = torch.randn((rows, 1104), device="cuda", generator=generator(13)).to(BF)
    x[1 << 16:] *= 100  # a sum taken from another turn's row would show
    w = torch.ones(1104, device="cuda")
    y, _, rstd = bfp8.rmsnorm(x, w)
    for at in (slice(0, 4000), slice(1 << 16, rows)):
        part = bfp8.rmsnorm(x[at], w)
        assert torch.equal(y[at], part[0]) and torch.equal(rstd[at], part[2])


@pytest.mark.parametrize("scales", ["fp32", "mx32"])
def test_codes_into_given_buffers(scales):
    """Codes in rows of a larger buffer: the same bytes, and nothing beside them."""
    x, residual, w, _ = inputs(256, 384, BF, 14, True)
    *want, r, rstd = bfp8.rmsnorm_quantize(x, w, residual, scales=scales, transposed=True)
    room = [torch.full((256, 512), 9, dtype=torch.uint8, device="cuda"),
            torch.full((384, 304), 9, dtype=torch.uint8, device="cuda")]
    s, st = (torch.empty_like(t) for t in (want[1], want[3]))
    total, stat = torch.empty_like(residual), torch.empty_like(rstd)
    out = bfp8.rmsnorm_quantize(x, w, residual, scales=scales, transposed=True, q=room[0][:, 64:448], s=s,
                                qt=room[1][:, 32:288], st=st, sum_out=total, rstd=stat)
    for a, b in zip(out, (*want, r, rstd)):
        assert torch.equal(a, b)
    assert torch.all(room[0][:, :64] == 9) and torch.all(room[0][:, 448:] == 9)
    assert torch.all(room[1][:, :32] == 9) and torch.all(room[1][:, 288:] == 9)
