"""float32 gates keep their digits however far they lie from zero, and bf16 ones give
the same bits.

With U = 2^-24: exp2 and the reciprocal are within one unit in the last place (2 U),
1 + rho takes two roundings and leaves rho^2 / 2 (rho under 4.9e-6 |g|: 2e-4 g^2 U),
the sum 1 + e is rounded once: sigma is within (7 + 2e-4 g^2) U, silu up within two
more.  Where sigma or a product is subnormal its last place, 2^-149, counts."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import U, f64, generator  # noqa: E402
from oracle import layer  # noqa: E402

LEAST = 2.0 ** -149


def gates():
    """Evenly over [-88.7, 88.7], and evenly in their logarithm."""
    gen = generator(21)
    even = (torch.rand(60000, device="cuda", generator=gen) * 2 - 1) * 88.7
    logs = torch.exp(torch.rand(20000, device="cuda", generator=gen) * 20 - 16) * even[:20000].sign()
    return torch.cat([even, logs.clamp(-88.7, 88.7)]).view(-1, 800)


def check(got, want, err):
    got = f64(got)
    worst = np.max(np.abs(got - want) / (err + 2 * LEAST))  # two products' last places
    assert np.all(np.isfinite(got)) and worst <= 1, worst


def test_values():
    g = gates()
    up = torch.randn(g.shape, device="cuda", generator=generator(22)) + 3
    h = layer.swiglu(f64(g), f64(up))
    x, u = np.abs(f64(g)), np.abs(f64(up))
    check(bfp8.swiglu(g, up), h, (9 + 2e-4 * x * x) * U * np.abs(h) + x * u * LEAST)


def test_gradient():
    """1 - sigma is within 3.5 U + 4 U (1 - sigma) for g > 0, and within one rounding
    and sigma's own error below; the sum, sigma and the products add 4 U."""
    g = gates()
    gen = generator(23)
    up, dh = (torch.randn(g.shape, device="cuda", generator=gen) for _ in range(2))
    dgate, dup = bfp8.swiglu_backward(dh, g, up)
    want, want_up = layer.swiglu_backward(f64(dh), f64(g), f64(up))
    x, a = f64(g), np.abs(f64(dh))
    s, o, q = layer._sigma(x), layer._sigma(-x), 2e-4 * x * x
    size = 1 + np.abs(x) * o
    err = s * U * ((19 + 2 * q) * size + 3.5 * np.maximum(x, 0)) + size * LEAST
    check(dgate, want, err * a * np.abs(f64(up)))
    check(dup, want_up, (9 + q) * U * np.abs(want_up) + np.abs(x) * a * LEAST)


def test_past_the_exponentials_range():
    """0 below -88.8, the gate itself above; so for the largest numbers."""
    g = torch.tensor([[-89.0, -200.0, -1e6, -3e38, 100.0, 1e6, 1e30, 3e38]], device="cuda")
    one = torch.ones_like(g)
    for dtype in (torch.float32, torch.bfloat16):
        gate = g.to(dtype)
        h = bfp8.swiglu(gate, one.to(dtype))
        assert torch.all(h[0, :4] == 0) and torch.equal(h[0, 4:], gate[0, 4:])
        dgate, dup = bfp8.swiglu_backward(one.to(dtype), gate, one.to(dtype))
        assert torch.all(dgate[0, :4] == 0) and torch.all(dgate[0, 4:] == 1)
        assert torch.all(dup[0, :4] == 0) and torch.equal(dup[0, 4:], gate[0, 4:])


@pytest.mark.parametrize("part", range(4))
def test_every_bf16_gate_gives_the_float32_bits(part):
    """All 2^16 patterns but NaN and infinity."""
    bits = torch.arange(part << 14, (part + 1) << 14, dtype=torch.int32, device="cuda").to(torch.int16)
    g = bits.view(torch.bfloat16)
    g = torch.where(torch.isfinite(g.float()), g, torch.zeros_like(g)).view(128, 128)
    one = torch.ones_like(g)
    for a, b in zip((bfp8.swiglu(g, one), *bfp8.swiglu_backward(one, g, one)),
                    (bfp8.swiglu(g.float(), one.float()),
                     *bfp8.swiglu_backward(one.float(), g.float(), one.float()))):
        assert torch.equal(a.view(torch.int16), b.to(torch.bfloat16).view(torch.int16))
    for a, b in zip(bfp8.swiglu_quantize(g, one, transposed=True),
                    bfp8.swiglu_quantize(g.float(), one.float(), transposed=True)):
        assert torch.equal(a, b)
