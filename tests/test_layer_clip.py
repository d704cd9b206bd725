"""The norm of many gradients and their clipping against float64.

The norm's squares are exact in float64 and its sum within 2^-40; the root is
rounded to float32: 2^-24 relative.  A clipped value is g times the float32
factor (norm, quotient and product: 3 roundings of 2^-24), then rounded."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import U, close, f64, generator  # noqa: E402
from oracle import layer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def check(grads, out, norm, max_norm):
    want = layer.grad_norm([f64(g) for g in grads])
    close(norm.reshape(1), np.array([want]), 1.1 * U * want)
    c = layer.clip_factor(want, max_norm)
    for g, o in zip(grads, out):
        close(o, f64(g) * c, 4 * U * np.abs(f64(g) * c), g.dtype)


@pytest.mark.parametrize("sizes", [[1], [1, 7, 8, 9], [16383, 16384, 16385, 3], [100000, 1, 70001],
                                   list(range(1, 120)), [3000001]])
@pytest.mark.parametrize("dtypes", [[BF], [F32], [BF, F32]])
@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
def test_clip(sizes, dtypes, max_norm):
    gen = generator(len(sizes))
    grads = [torch.randn(n, device="cuda", generator=gen).to(dtypes[i % len(dtypes)])
             for i, n in enumerate(sizes)]
    plan = bfp8.GradClip(grads, [torch.full_like(g, 9.0) for g in grads])
    norm = plan.clip(max_norm)
    check(grads, plan.out, norm, max_norm)
    before = [g.clone() for g in grads]
    again = bfp8.clip_grads(grads, max_norm)  # in place
    assert torch.equal(norm, again)
    for g, o, b in zip(grads, plan.out, before):
        assert torch.equal(g, o)
    assert torch.equal(norm, bfp8.grad_norm(before))
    # one call for both, or two: the same bits
    parts = bfp8.GradClip(before, [torch.empty_like(g) for g in grads])
    parts.clip(max_norm, norm=parts.norm())
    for o, p in zip(plan.out, parts.out):
        assert torch.equal(o, p)


@pytest.mark.parametrize("others", [False, True])  # a large tensor beside it or none
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lead,out_lead", [(0, 0), (1, 1), (3, 3), (1, 0), (0, 5), (2, 7)])
def test_any_alignment(dtype, lead, out_lead, others):
    n = 5003
    large = [torch.randn(300000, device="cuda", generator=generator(77)).to(dtype)] if others else []
    base = torch.randn(n + 16, device="cuda", generator=generator(lead)).to(dtype)
    room = torch.full((n + 16,), 9.0, dtype=dtype, device="cuda")
    g, o = base[lead:lead + n], room[out_lead:out_lead + n]
    clipped = [torch.empty_like(t) for t in large]
    norm = bfp8.clip_grads([g] + large, 1.0, out=[o] + clipped)
    check([g] + large, [o] + clipped, norm, 1.0)
    assert torch.all(room[:out_lead] == 9) and torch.all(room[out_lead + n:] == 9)


@pytest.mark.parametrize("others", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,ld,ldo", [(37, 100, 104, 104), (37, 100, 101, 128), (5, 2047, 2048, 2051),
                                              (300, 1, 3, 1), (1, 65, 200, 65), (64, 64, 64, 72)])
def test_strided(dtype, rows, cols, ld, ldo, others):
    large = [torch.randn(300000, device="cuda", generator=generator(78)).to(dtype)] if others else []
    base = torch.randn((rows, ld), device="cuda", generator=generator(ld)).to(dtype)
    room = torch.full((rows, ldo), 9.0, dtype=dtype, device="cuda")
    g, o = base[:, :cols], room[:, :cols]
    clipped = [torch.empty_like(t) for t in large]
    norm = bfp8.clip_grads([g] + large, 1.0, out=[o] + clipped)
    check([g] + large, [o] + clipped, norm, 1.0)
    assert torch.all(room[:, cols:] == 9)
    rest = base[:, cols:].clone()
    bfp8.clip_grads([g] + large, 1.0)
    assert torch.equal(g, o) and torch.equal(base[:, cols:], rest)


def test_more_sums_than_a_workgroup_adds_up():
    """Launches of up to 1024 partial sums each, more than 2048 in all: the norm has a
    launch of its own."""
    n = 1024 * 2048 * 4 // 64 + 5
    grads = [torch.randn(n, device="cuda", generator=generator(i)) for i in range(3 * 64)]
    plan = bfp8.GradClip(grads, [torch.empty_like(g) for g in grads])
    assert plan.workspace_bytes > 8 * 2048
    norm = plan.clip(1.0)
    want = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    assert abs(norm.item() - want.item()) <= 1.1 * U * want.item()
    for g, o in list(zip(grads, plan.out))[::50]:
        close(o, f64(g) / want.item(), 4 * U * np.abs(f64(g)) / want.item())


def test_sizes_that_float32_squares_lose():
    for scale, n in ((1e30, 5000), (1e-30, 5000), (1e30, 500000), (1e-30, 500000)):
        g = torch.randn(n, device="cuda", generator=generator(1)) * scale
        check([g], [g], bfp8.grad_norm([g]), float("inf"))
    g = torch.full((70000,), 1e-4, device="cuda")
    g[0] = 1e30
    check([g], [g], bfp8.grad_norm([g]), float("inf"))


def test_infinities_and_nan():
    for bad, norm_is, n in ((float("inf"), torch.isinf, 100), (float("nan"), torch.isnan, 100),
                            (float("inf"), torch.isinf, 200000), (float("nan"), torch.isnan, 200000)):
        g = torch.ones(n, device="cuda")
        g[3] = bad
        norm = bfp8.clip_grads([g], 1.0)
        assert norm_is(norm)
        assert torch.isnan(g[3])  # infinity times 0, or NaN
        rest = torch.cat([g[:3], g[4:]])
        assert torch.all(rest == 0) if bad == float("inf") else torch.all(torch.isnan(rest))
    g = torch.ones(100, device="cuda")
    bfp8.clip_grads([g], float("inf"))
    assert torch.all(g == 1)


def test_given_norm():
    """A norm over several ranks: their gradients as one set."""
    a, b = (torch.randn(999, device="cuda", generator=generator(s)) for s in (1, 2))
    norm = (bfp8.grad_norm([a]).square() + bfp8.grad_norm([b]).square()).sqrt()
    plan = bfp8.GradClip([a], [torch.empty_like(a)])
    assert plan.clip(2.0, norm=norm) is norm
    want = f64(a) * (2.0 / layer.grad_norm([f64(a), f64(b)]))
    close(plan.out[0], want, 8 * U * np.abs(want))


def test_zeros_empty_and_the_same_bits_again():
    zeros = [torch.zeros(10, device="cuda"), torch.empty(0, device="cuda")]
    assert bfp8.clip_grads(zeros, 1.0) == 0 and torch.all(zeros[0] == 0)
    assert bfp8.grad_norm([torch.empty(0, device="cuda")]) == 0
    grads = [torch.randn(n, device="cuda", generator=generator(n)) for n in (1 << 22, 77, 1 << 20)]
    norms = [bfp8.grad_norm(grads) for _ in range(5)]
    assert all(torch.equal(norms[0], n) for n in norms)
