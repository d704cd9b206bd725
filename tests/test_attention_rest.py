"""Rows that belong to no sequence (before cu[0], from cu[batch] on): the
results a call allocates are defined there (0, and -inf for lse), tensors that
are given keep what they hold unless the call is told to clear them."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

# name: (q lens, k lens, used keys or None, heads, kv heads, head size, rows before, rows after)
CASES = {
    "tiles": ([70, 0, 33], [70, 5, 40], None, 4, 2, 128, 3, 9),
    "head_40": ([20], [300], None, 3, 1, 40, 1, 0),
    "split": ([2600], [2600], None, 1, 1, 64, 2, 300),
    "streamed": ([1, 2], [2500, 2500], [2400, 7], 4, 2, 128, 5, 6),
    "no_rows_used": ([0], [0], None, 2, 2, 8, 10, 300),
    "much_padding": ([5], [5], None, 16, 8, 128, 0, 9000),
}


def make(name):
    q_lens, k_lens, used, H, KV, D, before, after = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(21)
    new = lambda T, h: torch.randn((T, h, D), device="cuda", generator=gen).to(torch.bfloat16)
    T, S = sum(q_lens) + before + after, sum(k_lens) + before + after
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = lambda lens: ints([before + sum(lens[:i]) for i in range(len(lens) + 1)])
    q, k, v, do = new(T, H), new(S, KV), new(S, KV), new(T, H)
    # rows of no sequence hold anything
    for t in (q, k, v, do):
        t[:before] = float("nan")
        t[t.shape[0] - after:] = float("inf")
    args = dict(cu_q=cu(q_lens), cu_k=cu(k_lens), k_lens=None if used is None else ints(used))
    return q, k, v, do, args, slice(before, T - after), slice(before, S - after)


def rest(t, rows):
    return torch.cat([t[:rows.start], t[rows.stop:]])


def dirty_pool(*shapes):
    """Memory that the next allocations of these sizes are likely to take."""
    for shape, dtype in shapes:
        torch.full(shape, 7.0, dtype=dtype, device="cuda")


@pytest.mark.parametrize("name", list(CASES))
def test_allocated_results_are_defined_everywhere(name):
    q, k, v, do, args, mine, keys = make(name)
    T, H, D = q.shape
    S, KV, _ = k.shape
    dirty_pool(((T, H, D), torch.bfloat16), ((H, T), torch.float32))
    o, lse = bfp8.attention_forward(q, k, v, **args)
    assert (rest(o, mine) == 0).all() and torch.isneginf(rest(lse.t(), mine)).all()
    dirty_pool(((T, H, D), torch.bfloat16), ((S, KV, D), torch.bfloat16),
               ((S, KV, D), torch.bfloat16))
    dq, dk, dv = bfp8.attention_backward(do, q, k, v, o, lse, **args)
    assert (rest(dq, mine) == 0).all()
    assert (rest(dk, keys) == 0).all() and (rest(dv, keys) == 0).all()
    # rows of sequences: as in tensors that are given
    new = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")
    o2, lse2, d2 = new(o), new(lse), [new(t) for t in (dq, dk, dv)]
    bfp8.attention_forward(q, k, v, **args, out=o2, lse=lse2)
    bfp8.attention_backward(do, q, k, v, o2, lse2, **args, dq=d2[0], dk=d2[1], dv=d2[2])
    for a, b, rows in ((o, o2, mine), (lse.t(), lse2.t(), mine), (dq, d2[0], mine),
                       (dk, d2[1], keys), (dv, d2[2], keys)):
        assert torch.equal(a[rows], b[rows]) and torch.isfinite(a[rows]).all()
        assert (rest(b, rows) == 7).all()


@pytest.mark.parametrize("name", list(CASES))
def test_given_results_are_cleared_when_asked(name):
    """Heads of wider rows, of which the others stay as they are."""
    q, k, v, do, args, mine, keys = make(name)
    wide = lambda t: torch.full((t.shape[0], t.shape[1] + 2, t.shape[2]), 7.0, dtype=t.dtype,
                                device="cuda")
    inner = lambda t: t[:, 1:-1]
    o, lse = wide(q), torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    bfp8.attention_forward(q, k, v, **args, out=inner(o), lse=lse, zero_rest=True)
    d = [wide(t) for t in (q, k, v)]
    bfp8.attention_backward(do, q, k, v, inner(o), lse, **args, dq=inner(d[0]), dk=inner(d[1]),
                            dv=inner(d[2]), zero_rest=True)
    assert torch.isneginf(rest(lse.t(), mine)).all()
    for t, rows in ((o, mine), (d[0], mine), (d[1], keys), (d[2], keys)):
        assert (rest(inner(t), rows) == 0).all() and torch.isfinite(t[rows]).all()
        assert (t[:, 0] == 7).all() and (t[:, -1] == 7).all()


def test_gradient_without_queries():
    """No query rows at all, keys of which some belong to no sequence."""
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((300, 2, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 0), device="cuda")
    dirty_pool((k.shape, k.dtype), (k.shape, k.dtype))
    dq, dk, dv = bfp8.attention_backward(q, q, k, k, q, lse, ints(0, 0, 0), ints(5, 200, 210))
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    new = [torch.full(k.shape, 7.0, dtype=k.dtype, device="cuda") for _ in range(2)]
    bfp8.attention_backward(q, q, k, k, q, lse, ints(0, 0, 0), ints(5, 200, 210), dk=new[0],
                            dv=new[1])
    for t in new:
        assert (t[5:210] == 0).all() and (t[:5] == 7).all() and (t[210:] == 7).all()


def test_each_result_by_itself():
    """A given tensor is left alone beside one that the call allocates."""
    q, k, v, do, args, mine, keys = make("tiles")
    T, H, D = q.shape
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    dirty_pool(((H, T), torch.float32))
    _, lse = bfp8.attention_forward(q, k, v, **args, out=o)
    assert (rest(o, mine) == 7).all() and torch.isneginf(rest(lse.t(), mine)).all()
    dk = torch.full(k.shape, 7.0, dtype=k.dtype, device="cuda")
    dirty_pool((q.shape, q.dtype), (v.shape, v.dtype))
    dq, _, dv = bfp8.attention_backward(do, q, k, v, o, lse, **args, dk=dk)
    assert (rest(dk, keys) == 7).all()
    assert (rest(dq, mine) == 0).all() and (rest(dv, keys) == 0).all()


def test_causal_is_a_truth_value():
    q = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    for causal in (2, 1 << 8, -1):
        with pytest.raises(ValueError, match="causal"):
            bfp8.attention_forward(q, q, q, causal=causal)


def test_clear_is_checked():
    """An unknown bit is refused before any HIP call."""
    h = bfp8.Heads(0x10000, 64, 64)
    for causal in (2, 1 << 7, 1 << 13, 1 | 1 << 14, -1):
        s = bfp8.AttentionShape(1, 4, 4, 0x10000, 0x10000, None, 1, 1, 64, causal, 0.125)
        assert bfp8.lib().bfp8_attention_forward(ctypes.byref(s), h, h, h, h, 0x10000, None, 0,
                                                 None) == 2
        assert bfp8.lib().bfp8_attention_workspace_bytes(ctypes.byref(s), 0) == \
            ctypes.c_size_t(-1).value
