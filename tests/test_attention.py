"""Attention and its gradient on the GPU against the float64 oracle, under the
element-wise bounds of oracle/attention.py."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

# name: (q lens, k lens, heads, kv heads, head size, causal, layout)
CASES = {
    "one_token": ([1], [1], 1, 1, 128, True, "dense"),
    "one_row_of_64": ([64], [64], 1, 1, 64, True, "dense"),
    "tile_edges": ([63, 64, 65], [63, 64, 65], 2, 2, 128, True, "fused"),
    "workgroup_edges": ([127, 128, 129], [127, 128, 129], 4, 2, 128, True, "fused"),
    "odd_group": ([86, 85, 171], [86, 85, 171], 6, 2, 64, True, "fused"),
    "eight_to_one": ([33, 32], [65, 100], 8, 1, 128, True, "heads"),
    "smallest_head": ([70], [70], 2, 1, 8, True, "dense"),
    "head_40": ([70, 3], [70, 200], 2, 1, 40, False, "fused_apart"),
    "head_80": ([130], [130], 2, 2, 80, True, "heads"),
    "head_104": ([65], [129], 4, 1, 104, False, "heads"),
    "cross": ([129, 200], [333, 77], 2, 2, 64, False, "heads"),
    "long_keys": ([5, 300], [700, 300], 2, 1, 128, True, "heads"),
    "empty_rows": ([200, 5, 300], [70, 4, 1], 4, 2, 128, True, "heads"),
    "empty_sequences": ([0, 5, 0, 0, 33, 0], [3, 5, 0, 9, 0, 0], 2, 1, 64, False, "heads"),
    "many_sequences": (list(range(70)), list(range(70)), 2, 1, 64, True, "fused"),
    "several_workgroups": ([700], [700], 2, 1, 128, True, "fused"),
}


def cu(lens):
    return [0] + [int(n) for n in np.cumsum(lens)]


def gpu_ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def tensors(T, S, H, KV, D, layout, gen):
    """q, k, v views in one of the layouts that the framework meets."""
    new = lambda *shape: torch.randn(shape, device="cuda", generator=gen).to(torch.bfloat16)
    if layout == "fused":  # the QKV projection's rows
        assert T == S
        rows = new(T, H + 2 * KV, D)
        return rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]
    if layout == "fused_apart":  # fused keys and values, row strides wider than the heads
        q, kv = new(T, H + 3, D), new(S, 2 * KV + 1, D)
        return q[:, 1:H + 1], kv[:, :KV], kv[:, KV:2 * KV]
    if layout == "heads":
        return new(H, T, D).transpose(0, 1), new(KV, S, D).transpose(0, 1), \
            new(KV, S, D).transpose(0, 1)
    return new(T, H, D), new(S, KV, D), new(S, KV, D)


def make(name, seed=0):
    q_lens, k_lens, H, KV, D, causal, layout = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = tensors(sum(q_lens), sum(k_lens), H, KV, D, layout, gen)
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    return q, k, v, do, cu(q_lens), cu(k_lens), causal, 1.0 / np.sqrt(D)


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, bound, what):
    """|got - want| <= bound wherever a result is due; an equal infinity is equal."""
    got = f64(got)
    due = ~np.isnan(want)
    assert not np.isnan(got[due]).any(), what
    same = got[due] == want[due]
    diff = np.abs(np.where(same, 0, got[due]) - np.where(same, 0, want[due]))
    # 1e-37: below bfloat16's smallest normal value
    ratio = (diff / (bound[due] + 1e-37)).max(initial=0.0)
    print(f"[bound] {what}: {ratio:.3f}", flush=True)
    assert ratio <= 1.0, (what, ratio)


@pytest.mark.parametrize("name", list(CASES))
def test_forward(name):
    q, k, v, _, cq, ck, causal, scale = make(name)
    o, lse = bfp8.attention_forward(q, k, v, gpu_ints(cq), gpu_ints(ck), causal=causal)
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), cq, ck, None, causal, scale)
    within(o, want, ob, name + " o")
    within(lse, wl, lb, name + " lse")


def backward(name, **kw):
    q, k, v, do, cq, ck, causal, scale = make(name)
    o, lse, *_ = ref.attention(f64(q), f64(k), f64(v), cq, ck, None, causal, scale)
    o = torch.tensor(o, device="cuda").to(torch.bfloat16)
    lse = torch.tensor(lse, device="cuda").float()
    grads = bfp8.attention_backward(do, q, k, v, o, lse, gpu_ints(cq), gpu_ints(ck), causal=causal,
                                    **kw)
    return grads, (q, k, v, do, cq, ck, causal, scale)


@pytest.mark.parametrize("name", list(CASES))
def test_backward(name):
    grads, (q, k, v, do, cq, ck, causal, scale) = backward(name)
    want = ref.attention_gradient(f64(do), f64(q), f64(k), f64(v), cq, ck, None, causal, scale)
    for i, n in enumerate(("dq", "dk", "dv")):
        within(grads[i], want[i], want[3 + i], f"{name} {n}")


@pytest.mark.parametrize("name", ["tile_edges", "head_40", "empty_rows", "long_keys"])
def test_backward_against_differences(name):
    """The gradients' products with random directions against central
    differences of the oracle's forward function."""
    grads, (q, k, v, do, cq, ck, causal, scale) = backward(name)
    x = [f64(t) for t in (q, k, v)]
    bounds = ref.attention_gradient(f64(do), *x, cq, ck, None, causal, scale)[3:]
    rng, step = np.random.default_rng(4), 1e-4
    for i, n in enumerate(("dq", "dk", "dv")):
        d = rng.choice([-1.0, 1.0], size=x[i].shape)
        f = lambda e: (ref.attention(*[t + e * d if j == i else t for j, t in enumerate(x)], cq, ck,
                                     None, causal, scale)[0] * f64(do)).sum()
        numeric = (f(step) - f(-step)) / (2 * step)
        # step^2 / 6 of a third derivative: at most a few per element and direction cubed
        slack = bounds[i].sum() + 1e-6 * abs(numeric) + 1e-3
        assert abs((f64(grads[i]) * d).sum() - numeric) <= slack, (n, numeric)


def test_equal_sequences_need_no_arrays():
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = tensors(3 * 50, 3 * 50, 4, 2, 64, "fused", gen)
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    at = gpu_ints([0, 50, 100, 150])
    o, lse = bfp8.attention_forward(q, k, v, batch=3)
    o2, lse2 = bfp8.attention_forward(q, k, v, at, at)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g, g2 = (bfp8.attention_backward(do, q, k, v, o, lse, **kw)
             for kw in (dict(batch=3), dict(cu_q=at, cu_k=at)))
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


@pytest.mark.parametrize("queries", [[1, 1, 1, 1, 1], [2, 1, 5, 1, 3], [40, 1, 90, 0, 7]])
@pytest.mark.parametrize("dim,heads,kv", [(128, 16, 8), (64, 4, 4), (80, 8, 1)])
def test_cache_with_room(queries, dim, heads, kv):
    """Sequences in a cache of fixed room: unused rows (NaN here), and rows
    of sequences without queries, have no part."""
    room, used = 700, [700, 1, 257, 64, 0]
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = tensors(sum(queries), room * 5, heads, kv, dim, "dense", gen)
    for b, n in enumerate(used):
        k[b * room + n:(b + 1) * room] = float("nan")
        v[b * room + n:(b + 1) * room] = float("nan")
    cq, ck = cu(queries), cu([room] * 5)
    scale = 1.0 / np.sqrt(dim)
    o, lse = bfp8.attention_forward(q, k, v, gpu_ints(cq), gpu_ints(ck), gpu_ints(used))
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), cq, ck, used, True, scale)
    within(o, want, ob, "o")
    within(lse, wl, lb, "lse")
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    o16 = torch.tensor(want, device="cuda").to(torch.bfloat16)
    grads = bfp8.attention_backward(do, q, k, v, o16, torch.tensor(wl, device="cuda").float(),
                                    gpu_ints(cq), gpu_ints(ck), gpu_ints(used))
    ref_g = ref.attention_gradient(f64(do), f64(q), f64(k), f64(v), cq, ck, used, True, scale)
    for i, n in enumerate(("dq", "dk", "dv")):
        within(grads[i], ref_g[i], ref_g[3 + i], n)


def test_single_queries_over_a_long_cache():
    """One query a sequence over thousands of keys, the keys split over
    workgroups: against the oracle, and the split against no split."""
    used = [4096, 3333, 1, 129]
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = tensors(4, 4096 * 4, 4, 2, 128, "dense", gen)
    cq, ck = cu([1] * 4), cu([4096] * 4)
    args = (q, k, v, gpu_ints(cq), gpu_ints(ck), gpu_ints(used))
    o, lse = bfp8.attention_forward(*args)
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), cq, ck, used, True, 128 ** -0.5)
    within(o, want, ob, "split o")
    within(lse, wl, lb, "split lse")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    o1, lse1 = bfp8.attention_forward(*args, workspace=small)
    within(o1, want, ob, "whole o")
    within(lse1, wl, lb, "whole lse")
    for _ in range(3):
        o2, lse2 = bfp8.attention_forward(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


STREAMED = {
    # name: (queries, used keys, room, heads, kv heads, head size, causal)
    "hundred_sequences": ([(1, 0, 2, 1)[i % 4] for i in range(100)],
                          [(i * 97) % 3300 for i in range(100)], 3300, 2, 1, 64, True),
    "many_rows": ([50, 1], [2500, 2000], 2500, 8, 2, 128, True),
    "not_causal": ([3, 40], [1, 1999], 2000, 4, 2, 80, False),
    "wide_group": ([1, 5], [1024, 1025], 1100, 16, 1, 128, True),
    "one_sequence": ([1], [5000], 5000, 1, 1, 128, True),
    "no_keys": ([2, 1, 1], [0, 1500, 0], 1500, 2, 2, 8, True),
    "no_queries": ([0, 3, 0, 0], [1500, 1400, 10, 0], 1500, 2, 2, 104, True),
    "more_queries_than_keys": ([40, 2], [7, 1200], 1200, 2, 1, 64, True),
}


@pytest.mark.parametrize("name", list(STREAMED))
def test_streamed_keys(name):
    """The kernel of few rows over many keys (it asks for a workspace), its
    joined parts, and the rows of no sequence left alone."""
    queries, used, room, H, KV, D, causal = STREAMED[name]
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, S = sum(queries) + 2, room * len(used)
    q, k, v = tensors(T, S, H, KV, D, "dense", gen)
    cq, ck = cu(queries), cu([room] * len(used))
    args = (q, k, v, gpu_ints(cq), gpu_ints(ck), gpu_ints(used))
    assert bfp8.attention_workspace_bytes(*args, causal=causal) > 0
    o = torch.full((T, H, D), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((H, T), 7.0, device="cuda")
    bfp8.attention_forward(*args, causal=causal, out=o, lse=lse)
    assert (o[-2:] == 7).all() and (lse[:, -2:] == 7).all()
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), cq, ck, used, causal, D ** -0.5)
    within(o, want, ob, name + " o")
    within(lse, wl, lb, name + " lse")
    o2, lse2 = bfp8.attention_forward(*args, causal=causal)
    assert torch.equal(o[:-2], o2[:-2]) and torch.equal(lse[:, :-2], lse2[:, :-2])


SPLIT = {
    # name: (q lens, k rows, used keys or None, heads, kv heads, head size, causal)
    "one_long": ([2000], [2000], None, 2, 1, 128, True),
    "ragged": ([30, 2600, 0, 700, 1], [30, 2600, 0, 700, 1], None, 2, 1, 64, True),
    "ragged_one_head": ([0, 2600, 30], [0, 2600, 30], None, 1, 1, 64, True),
    "cross": ([1900], [2500], None, 3, 1, 40, False),
    "empty_rows": ([2600], [2100], None, 2, 2, 128, True),
    "part_used": ([1500, 100], [2600, 2600], [2500, 1], 4, 1, 80, True),
}


@pytest.mark.parametrize("name", list(SPLIT))
def test_split_tiles(name):
    """Few workgroups over long sequences: long tiles' sums are split over
    several workgroups and added later, short ones are not, in one call."""
    q_lens, k_rows, used, H, KV, D, causal = SPLIT[name]
    gen = torch.Generator(device="cuda").manual_seed(12)
    T, S = sum(q_lens) + 3, sum(k_rows) + 2
    q, k, v = tensors(T, S, H, KV, D, "dense", gen)
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    cq, ck = cu(q_lens), cu(k_rows)
    args = (q, k, v, gpu_ints(cq), gpu_ints(ck), gpu_ints(used) if used else None)
    # "ragged" splits the gradients alone
    assert (bfp8.attention_workspace_bytes(*args, causal=causal) > 0) == (name != "ragged")
    assert bfp8.attention_workspace_bytes(*args, causal=causal, backward=True) > 8 * H * T + 16
    o = torch.full((T, H, D), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((H, T), 7.0, device="cuda")
    bfp8.attention_forward(*args, causal=causal, out=o, lse=lse)
    assert (o[-3:] == 7).all() and (lse[:, -3:] == 7).all()
    ref_args = (cq, ck, used, causal, D ** -0.5)
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), *ref_args)
    within(o, want, ob, name + " o")
    within(lse, wl, lb, name + " lse")
    whole, _ = bfp8.attention_forward(*args, causal=causal,
                                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    within(whole, want, ob, name + " o without a workspace")
    d = [torch.full(t.shape, 7.0, device="cuda", dtype=torch.bfloat16) for t in (q, k, v)]
    grads = bfp8.attention_backward(do, q, k, v, o, lse, *args[3:], causal=causal, dq=d[0], dk=d[1],
                                    dv=d[2])
    assert (d[0][-3:] == 7).all() and (d[1][-2:] == 7).all() and (d[2][-2:] == 7).all()
    ref_g = ref.attention_gradient(f64(do), f64(q), f64(k), f64(v), *ref_args)
    for i, n in enumerate(("dq", "dk", "dv")):
        within(grads[i], ref_g[i], ref_g[3 + i], f"{name} {n}")
    again = bfp8.attention_backward(do, q, k, v, o, lse, *args[3:], causal=causal)
    for a, b, rows in zip(grads, again, (T - 3, S - 2, S - 2)):
        assert torch.equal(a[:rows], b[:rows])


def test_scores_of_any_size():
    """Scores in the thousands (a running maximum that keeps growing, and one
    that starts at its largest), the same result for keys in either order."""
    n, D = 300, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = tensors(n, n, 2, 2, D, "dense", gen)
    k *= torch.linspace(0.1, 40, n, device="cuda")[:, None, None].to(torch.bfloat16)
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    for flip in (False, True):
        kk, vv = (t.flip(0) if flip else t for t in (k, v))
        o, lse = bfp8.attention_forward(q, kk, vv, causal=False, scale=2.0)
        want, wl, ob, lb = ref.attention(f64(q), f64(kk), f64(vv), [0, n], [0, n], None, False, 2.0)
        within(o, want, ob, "o")
        within(lse, wl, lb, "lse")
        grads = bfp8.attention_backward(do, q, kk, vv, o, lse, causal=False, scale=2.0)
        ref_g = ref.attention_gradient(f64(do), f64(q), f64(kk), f64(vv), [0, n], [0, n], None,
                                       False, 2.0)
        for i, m in enumerate(("dq", "dk", "dv")):
            within(grads[i], ref_g[i], ref_g[3 + i], m)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), torch.finfo(torch.bfloat16).min])
def test_sequences_do_not_touch_each_other(poison):
    """A poisoned sequence (and rows of no sequence) change nothing in its
    neighbours; rows and heads outside the views are not written."""
    lens = [100, 37, 60]
    gen = torch.Generator(device="cuda").manual_seed(9)
    H, KV, D, T = 4, 2, 64, sum(lens) + 13
    rows = torch.randn((T, H + 2 * KV, D), device="cuda", generator=gen).to(torch.bfloat16)
    at = gpu_ints([0, 100, 137, 197])
    do = torch.randn((T, H, D), device="cuda", generator=gen).to(torch.bfloat16)

    def both(rows, do):
        q, k, v = rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]
        o = torch.full((T, H + 1, D), 7.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((H, T), 7.0, device="cuda")
        bfp8.attention_forward(q, k, v, at, at, out=o[:, :H], lse=lse)
        d = torch.full((T, H + 2 * KV + 1, D), 7.0, device="cuda", dtype=torch.bfloat16)
        bfp8.attention_backward(do, q, k, v, o[:, :H], lse, at, at, dq=d[:, :H], dk=d[:, H:H + KV],
                                dv=d[:, H + KV:H + 2 * KV])
        assert (o[:, H] == 7).all() and (d[:, -1] == 7).all()
        assert (o[197:] == 7).all() and (lse[:, 197:] == 7).all() and (d[197:] == 7).all()
        return o, lse, d

    clean = both(rows, do)
    bad_rows, bad_do = rows.clone(), do.clone()
    bad_rows[100:137] = poison
    bad_rows[197:] = poison
    bad_do[100:137] = poison
    bad_do[197:] = poison
    bad = both(bad_rows, bad_do)
    for a, b in zip(clean, bad):
        a, b = (a, b) if a.dim() == 3 else (a.t(), b.t())
        for r in (slice(0, 100), slice(137, 197)):
            assert torch.equal(a[r], b[r])


def test_repeats_are_identical():
    q, k, v, do, cq, ck, causal, _ = make("several_workgroups")
    runs = []
    for _ in range(3):
        o, lse = bfp8.attention_forward(q, k, v, gpu_ints(cq), gpu_ints(ck), causal=causal)
        runs.append((o, lse) + bfp8.attention_backward(do, q, k, v, o, lse, gpu_ints(cq),
                                                       gpu_ints(ck), causal=causal))
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], run))


def test_offsets_past_32_bits():
    """Keys whose rows lie beyond 2^32 bytes of the cache's start, and a row
    stride near its largest: the last of 5 sequences of 300 rows of 2^21
    elements."""
    D, stride, n = 64, 1 << 21, 300
    gen = torch.Generator(device="cuda").manual_seed(10)
    room = torch.empty((5 * n, stride), dtype=torch.bfloat16, device="cuda")
    k = room[:, :D].view(5 * n, 1, D)
    v = room[:, stride - D:].view(5 * n, 1, D)
    k.copy_(torch.randn(k.shape, device="cuda", generator=gen))
    v.copy_(torch.randn(v.shape, device="cuda", generator=gen))
    q = torch.randn((5 * 20, 2, D), device="cuda", generator=gen).to(torch.bfloat16)
    cq, ck = cu([20] * 5), cu([n] * 5)
    o, lse = bfp8.attention_forward(q, k, v, gpu_ints(cq), gpu_ints(ck))
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), cq, ck, None, True, D ** -0.5)
    within(o, want, ob, "o")
    within(lse, wl, lb, "lse")
    do = torch.randn(q.shape, device="cuda", generator=gen).to(torch.bfloat16)
    grads = bfp8.attention_backward(do, q, k, v, o, lse, gpu_ints(cq), gpu_ints(ck))
    ref_g = ref.attention_gradient(f64(do), f64(q), f64(k), f64(v), cq, ck, None, True, D ** -0.5)
    for i, m in enumerate(("dq", "dk", "dv")):
        within(grads[i], ref_g[i], ref_g[3 + i], m)
    del room, k, v
    torch.cuda.empty_cache()


def test_runs_on_the_current_stream():
    q, k, v, do, cq, ck, causal, _ = make("workgroup_edges")
    at, ak = gpu_ints(cq), gpu_ints(ck)
    o, lse = bfp8.attention_forward(q, k, v, at, ak, causal=causal)
    want = (o, lse) + bfp8.attention_backward(do, q, k, v, o, lse, at, ak, causal=causal)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = bfp8.attention_forward(q, k, v, at, ak, causal=causal)
        got = (o, lse) + bfp8.attention_backward(do, q, k, v, o, lse, at, ak, causal=causal)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
