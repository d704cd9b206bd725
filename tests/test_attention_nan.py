"""NaN within a sequence's own rows: out of contract, but it does not pass for
a row that sees no key (L = -inf): L is NaN with O."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

# name: (queries, keys, heads, kv heads, head size): each joins its results in another place
CASES = {
    "tiles": (40, 70, 2, 1, 64),
    "split": (2600, 2600, 1, 1, 64),
    "streamed_whole": (1, 1100, 8, 8, 64),
    "streamed_joined": (2, 5000, 1, 1, 128),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("where", ["q", "k"])
def test_nan_scores_give_nan_lse(name, where):
    n, m, H, KV, D = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(41)
    new = lambda T, h: torch.randn((T, h, D), device="cuda", generator=gen).to(torch.bfloat16)
    q, k, v = new(n, H), new(m, KV), new(m, KV)
    (q if where == "q" else k)[0, 0, 3] = float("nan")  # the first key is seen by every query
    heads = slice(0, 1) if where == "q" else slice(0, H // KV)
    rows = slice(0, 1) if where == "q" else slice(0, n)
    o, lse = bfp8.attention_forward(q, k, v)
    assert torch.isnan(o[rows, heads]).all() and torch.isnan(lse[heads, rows]).all()
