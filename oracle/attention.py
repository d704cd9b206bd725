"""CPU reference of rotary positions, attention and attention's gradient, in
float64 from the definitions in include/bfp8_attention.h, one sequence and one
head at a time, with bounds on what the kernels' arithmetic may differ by.

Bounds.  u = 2^-8 is bfloat16's and w = 2^-24 float32's rounding error.  A
float32 sum of n products is off by at most 2 n w times the sum of their
magnitudes (the matrix core's order and inner rounding are left open).  So
  S      e_s = scale (2 D + 4) w sum|q||k|, and its exponential's argument
         adds 4 w (|S| + |L|) and the exponential itself 4 w: together e,
         the relative error of a probability;
  O      u |O| + (u + 2 e + 2 n w) sum p|v|  (P is rounded to bf16 once, the
         normaliser carries the same e and the sum over n keys);
  L      max e + 2 n w + 4 w |L|.
  dV     u |dV| + (u + e' + 2 n w) sum p|dO|, e' = e + the error of L;
  dS     p (|ddP| + |ddelta|) + (e' + u) |dS|, with |ddP| = 2 D w sum|dO||v|
         and |ddelta| = sum |dO| (u |O| + 2 D w |O|) for an O given in bf16;
  dQ     u |dQ| + scale sum (|ddS| + 2 n w |dS|)|k|, and dK alike.
"""

import numpy as np

U = 2.0 ** -8
W = 2.0 ** -24


def rope_angles(positions, rot, base=10000.0, scaling="none", factor=1.0, original=0):
    """(angles [T][rot/2], magnitude)"""
    out = np.zeros((len(positions), rot // 2))
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    magnitude = 0.1 * np.log(factor) + 1.0 if scaling == "yarn" else 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "yarn":
            turns = original * f / (2 * np.pi)
            g = min(max((turns - 1) / 31, 0.0), 1.0)
            f = g * f + (1 - g) * f / factor
        out[:, i] = np.asarray(positions, dtype=np.float64) * f
    return out, magnitude


def rope(x, positions, rot, layout="half", inverse=False, **kw):
    """x [T][H][D] -> the turned heads, by 2x2 matrices."""
    x = np.asarray(x, dtype=np.float64)
    angles, m = rope_angles(positions, rot, **kw)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = m * np.cos(angles[:, i])[:, None], m * np.sin(angles[:, i])[:, None]
        if inverse:  # the transposed matrix
            s = -s
        y[..., a] = c * x[..., a] - s * x[..., b]
        y[..., b] = s * x[..., a] + c * x[..., b]
    return y


def _sequences(cu_q, cu_k, k_lens):
    for b in range(len(cu_q) - 1):
        m = cu_k[b + 1] - cu_k[b]
        if k_lens is not None:
            m = min(m, k_lens[b])
        yield slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b] + m)


def _visible(n, m, causal):
    i, j = np.arange(n)[:, None], np.arange(m)[None]
    return j <= i + m - n if causal else np.ones((n, m), dtype=bool)


def _probabilities(q, k, scale, causal):
    """(P, S, L, e_s) of one head of one sequence; rows that see nothing have
    P = 0 and L = -inf."""
    vis = _visible(len(q), len(k), causal)
    s = np.where(vis, scale * (q @ k.T), -np.inf)
    top = s.max(1, initial=-np.inf, keepdims=True)
    p = np.exp(s - np.where(np.isinf(top), 0, top))
    total = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.log(total) + np.where(np.isinf(top), 0, top))[:, 0]
    p = p / np.where(total > 0, total, 1)
    e = scale * (2 * q.shape[1] + 4) * W * (np.abs(q) @ np.abs(k).T)
    finite = np.where(np.isinf(lse), 0, lse)[:, None]
    e = e + 4 * W * (np.abs(np.where(vis, s, 0)) + np.abs(finite)) + 4 * W
    return p, lse, np.where(vis, e, 0)


def attention(q, k, v, cu_q, cu_k, k_lens, causal, scale):
    """(o, lse, bound of o, bound of lse); rows of no sequence are NaN."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    group = q.shape[1] // k.shape[1]
    o, ob = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, lb = np.full((q.shape[1], len(q)), np.nan), np.full((q.shape[1], len(q)), np.nan)
    for r, c in _sequences(cu_q, cu_k, k_lens):
        for h in range(q.shape[1]):
            g = h // group
            p, L, e = _probabilities(q[r, h], k[c, g], scale, causal)
            n = p.shape[1]
            o[r, h] = p @ v[c, g]
            worst = e.max(1, initial=0.0)
            weight = (p * (U + 2 * worst[:, None] + 2 * n * W)) @ np.abs(v[c, g])
            ob[r, h] = U * np.abs(o[r, h]) + weight
            lse[h, r] = L
            lb[h, r] = worst + 2 * n * W + 4 * W * np.abs(np.where(np.isinf(L), 0, L))
    return o, lse, ob, lb


def attention_gradient(dout, q, k, v, cu_q, cu_k, k_lens, causal, scale):
    """(dq, dk, dv) and their bounds, for kernels given O rounded to bf16 and
    L in float32; rows of no sequence are NaN, unused key rows 0."""
    dout, q, k, v = (np.asarray(t, dtype=np.float64) for t in (dout, q, k, v))
    group = q.shape[1] // k.shape[1]
    dq, bq = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    out = [np.full(k.shape, np.nan) for _ in range(4)]
    for b in range(len(cu_q) - 1):
        for t in out:
            t[cu_k[b]:cu_k[b + 1]] = 0.0
    dk, dv, bk, bv = out
    D = q.shape[2]
    for r, c in _sequences(cu_q, cu_k, k_lens):
        for h in range(q.shape[1]):
            g = h // group
            p, L, e = _probabilities(q[r, h], k[c, g], scale, causal)
            do = dout[r, h]
            o = p @ v[c, g]
            dp = do @ v[c, g].T
            ds = p * (dp - (do * o).sum(1, keepdims=True))
            e = e + e.max(1, initial=0.0)[:, None] + 2 * p.shape[1] * W
            ddp = 2 * D * W * (np.abs(do) @ np.abs(v[c, g]).T)
            ddelta = (np.abs(do) * np.abs(o)).sum(1, keepdims=True) * (U + 2 * D * W)
            dds = p * (ddp + ddelta) + (e + U) * np.abs(ds)
            dq[r, h] = scale * (ds @ k[c, g])
            bq[r, h] = U * np.abs(dq[r, h]) + scale * (
                (dds + 2 * p.shape[1] * W * np.abs(ds)) @ np.abs(k[c, g]))
            dk[c, g] += scale * (ds.T @ q[r, h])
            bk[c, g] += scale * ((dds + 2 * group * len(ds) * W * np.abs(ds)).T @ np.abs(q[r, h]))
            dv[c, g] += p.T @ do
            bv[c, g] += (p * (U + e + 2 * group * len(ds) * W)).T @ np.abs(do)
    return dq, dk, dv, bq, bk + U * np.abs(dk), bv + U * np.abs(dv)
