"""The attention block where the sequences leave rows of the pass unused (a
micro-batch padded to its size): whatever those rows hold, they are no part of
any result, in every pass."""
import pytest
import torch

import test_attention_block as base

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from blockwise_fp8_gemm_bfp8_amd.attention_block import AttentionBlock  # noqa: E402

TOKENS = 384
HEADS, KV, D, HIDDEN = base.HEADS, base.KV, base.D, base.HIDDEN


def make(lens, before, seed, padding_position=0):
    """A block of 384 tokens whose sequences start after `before` rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda shape, std: (torch.randn(shape, device="cuda", generator=gen) * std).to(torch.bfloat16)
    starts = [before + sum(lens[:i]) for i in range(len(lens) + 1)]
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    positions = torch.full((TOKENS,), padding_position, dtype=torch.int32)
    for a, n in zip(starts, lens):
        positions[a:a + n] = torch.arange(n, dtype=torch.int32)
    w_qkv, w_o = new(((HEADS + 2 * KV) * D, HIDDEN), 0.05), new((HIDDEN, HEADS * D), 0.05)
    block = AttentionBlock(w_qkv, w_o, HEADS, KV, TOKENS, cu, positions.cuda(),
                           bfp8.rope_table(TOKENS, D))
    block.quantize_weights()
    return block, new((TOKENS, HIDDEN), 1.0), new((TOKENS, HIDDEN), 1e-3), slice(before, starts[-1])


def poison(block, value):
    for name in ("a", "lse", "qkv", "dqkv", "da"):
        block.buf[name].fill_(value)


def reference(block, x, dy, rows, lens, monkeypatch):
    """Autograd over the rows of sequences alone."""
    monkeypatch.setattr(base, "LENS", lens)
    positions, block.positions = block.positions, block.positions[rows]
    try:
        y, dx, dw_qkv, dw_o = base.reference(block, x[rows], dy[rows])
    finally:
        block.positions = positions
    return y, dx, dw_qkv, dw_o


@pytest.mark.parametrize("value", [float("nan"), 1e4])
@pytest.mark.parametrize("lens,before", [([200, 1, 60], 0), ([130, 7], 40)])
def test_padded_block_matches_autograd(lens, before, value, monkeypatch):
    """The bound of the full block (15 %): leftovers in the unused rows are off
    by orders of magnitude or NaN."""
    block, x, dy, rows = make(lens, before, 3)
    want = reference(block, x, dy, rows, lens, monkeypatch)
    for _ in range(2):
        poison(block, value)
        y = block.forward(x)
        dx, dw_qkv, dw_o = block.backward(dy)
        got = (y[rows], dx[rows], dw_qkv, dw_o)
        for name, a, b in zip(("y", "dx", "dw_qkv", "dw_o"), got, want):
            err = ((a.float() - b).norm() / b.norm()).item()
            print(f"[block] {name}: {err:.4f}", flush=True)
            assert err < 0.15, (name, err)
        for t in (y, dx):
            assert (t[:rows.start] == 0).all() and (t[rows.stop:] == 0).all()


def test_unused_rows_change_nothing():
    """Leftovers, and positions outside the table on the unused rows (the usual
    mark of padding), change no bit."""
    block, x, dy, rows = make([200, 1, 60], 0, 4)
    poison(block, 0.0)
    y = block.forward(x).clone()
    want = [y] + [t.clone() for t in block.backward(dy)]
    other, *_ = make([200, 1, 60], 0, 4, padding_position=-1)
    poison(other, float("nan"))
    for _ in range(2):
        y = other.forward(x)
        for a, b in zip([y, *other.backward(dy)], want):
            assert torch.equal(a, b)


def test_sequences_change_between_passes():
    """The next micro-batch's starts and positions in the same device arrays,
    fewer rows used than before."""
    block, x, dy, _ = make([200, 100, 84], 0, 5)
    block.forward(x)
    block.backward(dy)
    fresh, *_ = make([150, 10, 3], 0, 5)
    block.cu.copy_(fresh.cu)
    block.positions.copy_(fresh.positions)
    poison(fresh, 0.0)
    for a, b in zip([block.forward(x), *block.backward(dy)], [fresh.forward(x), *fresh.backward(dy)]):
        assert torch.equal(a, b)


def test_default_positions_past_the_table():
    """Without positions token t stands at t; the unused rows may stand past the
    table's end."""
    block, x, dy, _ = make([200], 0, 6)
    y = block.forward(x).clone()
    want = [y] + [t.clone() for t in block.backward(dy)]
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    other = AttentionBlock(block.w_qkv, block.w_o, HEADS, KV, TOKENS, cu, None,
                           bfp8.rope_table(200, D))
    other.quantize_weights()
    poison(other, float("nan"))
    y = other.forward(x)
    for a, b in zip([y, *other.backward(dy)], want):
        assert torch.equal(a, b)


def test_graph_replays_take_the_current_sequences():
    """Captured once, replayed over micro-batches of different lengths."""
    block, x, dy, _ = make([200, 100, 84], 0, 7)
    eager, *_ = make([200, 100, 84], 0, 7)
    block.forward(x)
    block.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x)
        block.backward(dy)
    for lens, before in (([200, 1, 60], 0), ([10, 300, 74], 0), ([5, 6, 7], 300)):
        fresh, *_ = make(lens, before, 7)
        for b in (block, eager):
            b.cu.copy_(fresh.cu)
            b.positions.copy_(fresh.positions)
        torch.cuda.synchronize()
        graph.replay()
        want = [eager.forward(x), *eager.backward(dy)]
        torch.cuda.synchronize()
        for name, b in zip(("y", "dx", "dw_qkv", "dw_o"), want):
            assert torch.equal(block.buf[name], b), name
