"""The attention oracle against what does not share its formulas: torch's
float64 autograd through an explicit softmax, central differences, complex
multiplication, and hand-made cases."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

CASES = [
    # (q lens, k lens, heads, kv heads, dim, causal)
    ([5], [5], 2, 1, 8, True),
    ([1, 4, 0, 3], [7, 4, 2, 0], 4, 2, 8, True),
    ([6], [3], 2, 2, 16, True),       # the first rows see nothing
    ([3, 2], [4, 9], 3, 1, 8, False),
]


def draw(q_lens, k_lens, H, KV, D, seed=0):
    rng = np.random.default_rng(seed)
    cu = lambda lens: [0] + list(np.cumsum(lens))
    q = rng.normal(size=(sum(q_lens), H, D))
    k, v = rng.normal(size=(2, sum(k_lens), KV, D))
    return q, k, v, rng.normal(size=q.shape), cu(q_lens), cu(k_lens)


def library(q, k, v, cu_q, cu_k, causal, scale):
    rows, group = [], q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        qs = q[cu_q[b]:cu_q[b + 1]].transpose(0, 1)
        ks = k[cu_k[b]:cu_k[b + 1]].transpose(0, 1).repeat_interleave(group, 0)
        vs = v[cu_k[b]:cu_k[b + 1]].transpose(0, 1).repeat_interleave(group, 0)
        s = qs @ ks.transpose(1, 2) * scale
        if causal:
            seen = torch.ones((n, m), dtype=torch.bool).tril(m - n)
            s = torch.where(seen, s, torch.tensor(-1e30, dtype=s.dtype))
            p = torch.softmax(s, -1) * seen if m else s
        else:
            p = torch.softmax(s, -1)
        rows.append((p @ vs).transpose(0, 1))
    return torch.cat(rows)


@pytest.mark.parametrize("case", CASES)
def test_attention_and_gradient_match_autograd(case):
    q_lens, k_lens, H, KV, D, causal = case
    q, k, v, do, cu_q, cu_k = draw(q_lens, k_lens, H, KV, D)
    scale = 0.37
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    o = library(*t, cu_q, cu_k, causal, scale)
    grads = torch.autograd.grad((o * torch.tensor(do)).sum(), t)
    got, lse, ob, lb = ref.attention(q, k, v, cu_q, cu_k, None, causal, scale)
    np.testing.assert_allclose(got, o.detach().numpy(), atol=1e-12)
    assert (ob >= 0).all() and (lb >= 0).all()
    out = ref.attention_gradient(do, q, k, v, cu_q, cu_k, None, causal, scale)
    for have, want in zip(out, grads):
        np.testing.assert_allclose(have, want.numpy(), atol=1e-12)


@pytest.mark.parametrize("case", CASES)
def test_gradient_matches_differences(case):
    q_lens, k_lens, H, KV, D, causal = case
    q, k, v, do, cu_q, cu_k = draw(q_lens, k_lens, H, KV, D, seed=1)
    grads = ref.attention_gradient(do, q, k, v, cu_q, cu_k, None, causal, 0.5)[:3]
    rng, step = np.random.default_rng(2), 1e-5
    for i, grad in enumerate(grads):
        if grad.size == 0:
            continue
        d = rng.normal(size=grad.shape)
        f = lambda e: (ref.attention(*[x + e * d if j == i else x for j, x in
                                       enumerate((q, k, v))], cu_q, cu_k, None, causal,
                                     0.5)[0] * do).sum()
        # central difference: error step^2 times a third derivative of order one
        assert abs((f(step) - f(-step)) / (2 * step) - (grad * d).sum()) < 1e-6


def test_rows_that_see_nothing_and_unused_keys():
    q, k, v, do, cu_q, cu_k = draw([6, 2], [3, 5], 2, 1, 8)
    o, lse, _, _ = ref.attention(q, k, v, cu_q, cu_k, [3, 0], True, 1.0)
    assert (o[:3] == 0).all() and np.isneginf(lse[:, :3]).all() and np.isfinite(lse[:, 3:6]).all()
    np.testing.assert_allclose(o[3], v[0, 0][None].repeat(2, 0))  # one visible key
    assert (o[6:] == 0).all()
    dq, dk, dv, *_ = ref.attention_gradient(do, q, k, v, cu_q, cu_k, [3, 0], True, 1.0)
    assert (dq[:3] == 0).all() and (dk[3:] == 0).all() and (dv[3:] == 0).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_complex_product(layout):
    rng = np.random.default_rng(3)
    x, rot, pos = rng.normal(size=(7, 2, 12)), 8, [0, 1, 5, 2, 1000, 7, 3]
    y = ref.rope(x, pos, rot, layout, base=100.0)
    a = x[..., :4] if layout == "half" else x[..., 0:8:2]
    b = x[..., 4:8] if layout == "half" else x[..., 1:8:2]
    f = 100.0 ** (-np.arange(4) / 4.0)
    z = (a + 1j * b) * np.exp(1j * np.asarray(pos)[:, None, None] * f)
    got = (y[..., :4] + 1j * y[..., 4:8]) if layout == "half" else y[..., 0:8:2] + 1j * y[..., 1:8:2]
    np.testing.assert_allclose(got, z, atol=1e-12)
    assert (y[..., 8:] == x[..., 8:]).all()
    # the gradient of a turn is its transpose: here its inverse
    np.testing.assert_allclose(ref.rope(y, pos, rot, layout, inverse=True, base=100.0), x, atol=1e-12)


def test_rope_scalings():
    pos = [4096]
    plain, m = ref.rope_angles(pos, 64)
    assert m == 1.0 and plain[0, 0] == 4096
    np.testing.assert_allclose(ref.rope_angles(pos, 64, scaling="linear", factor=4.0)[0], plain / 4)
    ntk = ref.rope_angles(pos, 64, scaling="ntk", factor=4.0)[0]
    # the fastest pair stays, the slowest is interpolated by the whole factor
    np.testing.assert_allclose([ntk[0, 0] / plain[0, 0], ntk[0, -1] / plain[0, -1]], [1.0, 0.25])
    yarn, m = ref.rope_angles(pos, 64, scaling="yarn", factor=4.0, original=4096)
    assert abs(m - (0.1 * np.log(4.0) + 1)) < 1e-15
    ratio = yarn / plain
    turns = plain[0] / (2 * np.pi)
    assert np.allclose(ratio[0][turns > 32], 1.0) and np.allclose(ratio[0][turns < 1], 0.25)
    assert (np.diff(ratio[0]) <= 1e-15).all()


def test_rounding_units():
    """U and W are the largest relative errors of rounding to nearest in
    bfloat16 (8 significant bits) and float32 (24): met at the midpoint above
    a power of two, never passed."""
    mid = torch.tensor([1 + 2.0 ** -8], dtype=torch.float64)
    assert abs(mid.to(torch.bfloat16).double() - mid) == ref.U
    x = torch.rand(100000, dtype=torch.float64, generator=torch.Generator().manual_seed(0)) + 1
    err = (x.to(torch.bfloat16).double() - x).abs() / x
    assert 0.9 * ref.U < err.max() <= ref.U
    assert ((x.float().double() - x).abs() / x).max() <= ref.W
