"""Rotary positions on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

W = 2.0 ** -24
SCALINGS = [("none", 1.0, 0), ("linear", 2.0, 0), ("ntk", 4.0, 0), ("yarn", 8.0, 512)]


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("scaling,factor,original", SCALINGS)
@pytest.mark.parametrize("rot", [2, 64, 128])
def test_table(scaling, factor, original, rot):
    n = 70001
    table = bfp8.rope_table(n, rot, 10000.0, scaling, factor, original)
    pos = [0, 1, 2, 511, 4096, n - 1]
    angles, m = ref.rope_angles(pos, rot, 10000.0, scaling, factor, original)
    want = m * np.stack([np.cos(angles), np.sin(angles)], -1)
    # one rounding to float32, and angles that two float64 programs give within 1e-10
    assert np.abs(f64(table)[pos] - want).max() <= m * (W + 1e-9)


def turned(x, table, pos, rot, layout, inverse, kw):
    want = ref.rope(f64(x), f64(pos), rot, layout, inverse, **kw)
    got = f64(bfp8.rope(x, table, pos, layout=layout, inverse=inverse))
    # two rounded products of a rounded cosine and sine, their sum, and the output's rounding
    out = ref.U if x.dtype == torch.bfloat16 else W
    size = np.abs(f64(x)).max() * 2 * 1.5
    assert (np.abs(got - want) <= out * np.abs(want) + 6 * W * size).all()
    assert (got[..., rot:] == f64(x)[..., rot:]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 8, 2), (3, 5, 128, 128), (257, 24, 128, 128),
                                       (33, 3, 80, 32), (17, 2, 80, 40), (9, 7, 72, 48),
                                       (5, 1, 96, 64), (7, 2, 40, 14), (4, 3, 256, 256),
                                       (2, 1, 512, 510)])
def test_rope(layout, inverse, dtype, T, H, D, rot):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H + 1, D), device="cuda", generator=gen).to(dtype)[:, 1:]
    kw = dict(scaling="yarn", factor=4.0, original=256)
    table = bfp8.rope_table(3000, rot, 10000.0, "yarn", 4.0, 256)
    pos = torch.randint(0, 3000, (T,), device="cuda", generator=gen, dtype=torch.int32)
    turned(x, table, pos, rot, layout, inverse, kw)


def test_default_positions_in_place_and_head_major():
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = bfp8.rope_table(100, 32)
    x = torch.randn((4, 100, 64), device="cuda", generator=gen).to(torch.bfloat16).transpose(0, 1)
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    want = bfp8.rope(x, table, pos)
    assert torch.equal(bfp8.rope(x, table), want)
    rows = torch.randn((100, 6, 64), device="cuda", generator=gen).to(torch.bfloat16)
    want, before = bfp8.rope(rows[:, :4], table, pos), rows.clone()
    assert bfp8.rope(rows[:, :4], table, pos, out=rows[:, :4]).data_ptr() == rows.data_ptr()
    assert torch.equal(rows[:, :4], want) and torch.equal(rows[:, 4:], before[:, 4:])


def test_gradient_is_the_transpose():
    """<rope(x), g> = <x, rope(g, inverse)> for a linear map and its gradient,
    and the difference quotient of a linear map is the map."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    table = bfp8.rope_table(50, 64, scaling="yarn", factor=4.0, original_length=64)
    x, g, d = torch.randn((3, 50, 3, 96), device="cuda", generator=gen)
    for layout in ("half", "interleaved"):
        y = bfp8.rope(x, table, layout=layout)
        dx = bfp8.rope(g, table, layout=layout, inverse=True)
        a, b = (f64(y) * f64(g)).sum(), (f64(x) * f64(dx)).sum()
        size = (np.abs(f64(y)) * np.abs(f64(g))).sum() * 2
        assert abs(a - b) <= 8 * W * size
        diff = bfp8.rope(x + d, table, layout=layout) - y
        assert abs((f64(diff) * f64(g)).sum() - (f64(d) * f64(dx)).sum()) <= 32 * W * size


def test_positions_outside_the_table_give_nan():
    table = bfp8.rope_table(10, 16)
    x = torch.ones((4, 2, 32), device="cuda", dtype=torch.bfloat16)
    y = bfp8.rope(x, table, torch.tensor([9, 10, -1, 0], dtype=torch.int32, device="cuda"))
    assert torch.isfinite(y[[0, 3]]).all() and (y[:, :, 16:] == 1).all()
    assert torch.isnan(y[1:3, :, :16]).all()


def test_large_tensor_offsets():
    """Rows past 2^32 bytes."""
    T, row = 1030, 1 << 22
    room = torch.empty((T, row), dtype=torch.bfloat16, device="cuda")
    x = room[:, :64].view(T, 1, 64)
    x.fill_(1.0)
    table = bfp8.rope_table(T, 64)
    y = bfp8.rope(x, table)
    assert torch.equal(y, bfp8.rope(x.contiguous(), table))
    del room, x
    torch.cuda.empty_cache()
