"""The norm's statistics: rows whose squares' sum passes float32 although their mean does
not, and how exact the reciprocal root is.  U = 2^-24."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import EPS, U, check_codes, close, f64, generator, padded  # noqa: E402
from oracle import layer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NORM = 32 * U  # as in the tests of ordinary rows


def huge_rows(rows, cols, dtype, seed):
    """Ordinary rows and rows of mean squares up to 2^127 in turn; one has all of it in
    one value."""
    gen = generator(seed)
    x = padded(rows, cols, dtype, gen, 1.0, 1)
    scale = torch.tensor([1.0, 3e18, 9e18, 1e-3, 4e17], device="cuda").repeat(-(-rows // 5))[:rows]
    x.copy_((x.float() * scale[:, None]).to(dtype))
    x[rows - 1] = 1.0
    x[rows - 1, cols // 2] = -1.2e19 * cols ** 0.5
    want = f64(x)
    mean = np.mean(want * want, axis=1)
    assert np.all(np.isfinite(want)) and np.all(mean < 2.0 ** 127.9)
    assert np.sum(mean * cols > 2.0 ** 128) >= 2 or cols < 4
    return x


@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(23, 2), (40, 100), (11, 500), (13, 1000), (9, 2048), (7, 4000),
                                       (6, 8192), (12, 16384)])
def test_huge_rows(rows, cols, dtype, added):
    x = huge_rows(rows, cols, dtype, cols)
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=generator(1))
    residual = padded(rows, cols, dtype, generator(7), 0.0) if added else None
    y, r, rstd = bfp8.rmsnorm(x, w, residual, eps=EPS)
    want, stat = layer.rmsnorm(f64(x), f64(w), EPS)
    close(rstd, stat, NORM * stat)
    close(y, want, NORM * np.abs(want), dtype)
    dy = padded(rows, cols, dtype, generator(2), 1.0)
    dx, dw = bfp8.rmsnorm_backward(dy, r, w, rstd)
    want_dx, want_dw = layer.rmsnorm_backward(f64(dy), f64(x), f64(w), EPS)
    t, g = np.abs(f64(x) * stat[:, None]), np.abs(f64(dy) * f64(w))
    err = 64 * U * stat[:, None] * (g + t * np.mean(g * t, axis=1)[:, None])
    close(dx, want_dx, err, dtype)
    close(dw, want_dw, 140 * U * np.sum(np.abs(f64(dy)) * t, axis=0))


@pytest.mark.parametrize("cols", [128, 2048, 16384])
def test_codes_of_huge_rows(cols):
    x = huge_rows(128, cols, BF, cols + 1)
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=generator(3))
    *out, _, rstd = bfp8.rmsnorm_quantize(x, w, eps=EPS, transposed=True)
    want, stat = layer.rmsnorm(f64(x), f64(w), EPS)
    close(rstd, stat, NORM * stat)
    check_codes(out, want, NORM * np.abs(want), "fp32")


def test_more_huge_rows_than_workgroups():
    """Every turn's second sum is its own."""
    rows = (1 << 16) + 500
    x = torch.randn((rows, 520), device="cuda", generator=generator(4)) * 1.1e19
    x[1 << 16:] *= 0.5
    w = torch.ones(520, device="cuda")
    y, _, rstd = bfp8.rmsnorm(x, w)
    for at in (slice(0, 600), slice(1 << 16, rows)):
        part = bfp8.rmsnorm(x[at], w)
        assert torch.equal(y[at], part[0]) and torch.equal(rstd[at], part[2])
    stat = (x[-600:].double().square().mean(1) + 1e-6).rsqrt()
    close(rstd[-600:], f64(stat), NORM * f64(stat))


def test_infinity_and_nan_stay_in_their_rows():
    x = torch.randn((6, 700), device="cuda", generator=generator(5))
    w = torch.ones(700, device="cuda")
    clean = bfp8.rmsnorm(x, w)
    bad = x.clone()
    bad[1, 3], bad[4, 600] = float("inf"), float("nan")
    y, _, rstd = bfp8.rmsnorm(bad, w)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(rstd[keep], clean[2][keep])
    assert torch.isnan(y[1, 3]) and torch.all(torch.isnan(y[4]))


@pytest.mark.parametrize("cols", [1020, 2048, 8160, 16372, 16380])
def test_the_reciprocal_root_of_an_exact_sum(cols):
    """Integers whose squares add up exactly: what is left is one rounding of mean + eps
    (half of U in the root), one of its product with the estimate (half of U again), and the
    last one: 2 U.  (The estimate's own 2 U are squared away.)"""
    rows = 20000
    gen = generator(6)
    x = torch.randint(-4, 5, (rows, cols), device="cuda", generator=gen).float()
    x[:, 0] = torch.arange(rows, device="cuda") % 1000
    exact = x.double().square().sum(1)
    assert torch.all(exact < 2 ** 24)
    _, _, rstd = bfp8.rmsnorm(x, torch.ones(cols, device="cuda"), eps=EPS)
    want = (exact / cols + float(np.float32(EPS))).rsqrt()
    worst = ((rstd.double() - want).abs() / want).max().item() / U
    print(f"[norm] {cols}: {worst:.2f}", flush=True)
    assert worst <= 2.0, worst
