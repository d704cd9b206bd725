"""A pair of zeros turned by any angle is zero, also at a position outside the
table, where other values become NaN."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,D", [(128, 128), (64, 96), (24, 40), (14, 40)])
def test_zero_pairs_outside_the_table(rot, D, dtype, layout, inverse):
    gen = torch.Generator(device="cuda").manual_seed(61)
    table = bfp8.rope_table(10, rot)
    x = torch.randn((6, 3, D), device="cuda", generator=gen).to(dtype)
    x[2:4] = 0.0
    x[2, 1] = -0.0
    x[4, 0, 0] = 0.0  # one of a pair: not a zero pair
    a, b = (0, rot // 2) if layout == "half" else (0, 1)
    x[5, 2, a] = x[5, 2, b] = 0.0
    pos = torch.tensor([9, -1, -1, 10, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    for out in (None, x.clone()):
        if out is None:
            y = bfp8.rope(x, table, pos, layout=layout, inverse=inverse)
        else:
            y = bfp8.rope(out, table, pos, layout=layout, inverse=inverse, out=out)
        assert torch.isfinite(y[0]).all() and (y[2:4] == 0).all()
        nan = torch.isnan(y[[1, 4, 5], :, :rot])
        assert nan[:2].all() and nan[2, :2].all()
        want = torch.ones(rot, dtype=torch.bool, device="cuda")
        want[[a, b]] = False
        assert torch.equal(nan[2, 2], want) and (y[5, 2, [a, b]] == 0).all()
        assert torch.equal(y[..., rot:], x[..., rot:])
