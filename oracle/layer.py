"""What a decoder layer computes around its linears, in float64 from the
formulas: the RMS norm with the residual's addition, the gated activation, their
gradients, the global norm of gradients and clipping; and how far E4M3 codes and
scales of a computed result may be from those of the exact one.

The norm is of the stored sum (rounded to the tensors' type): callers pass that.
"""

import numpy as np

from .e4m3 import E4M3_MAX, e4m3_decode, e4m3_encode


def rmsnorm(r, w, eps):
    """(y, rstd) of rows r, in float64."""
    r, w = np.asarray(r, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, r, w, eps, dsum=None):
    """(dx, dw): the derivative of sum(dy * y) (+ sum(dsum * r)) by r and w."""
    dy, r, w = (np.asarray(t, np.float64) for t in (dy, r, w))
    _, rstd = rmsnorm(r, w, eps)
    n = r.shape[1]
    # y_j = w_j r_j s, ds/dr_i = -s^3 r_i / n
    through = np.sum(dy * w * r, axis=1) * rstd ** 3 / n
    dx = dy * w * rstd[:, None] - r * through[:, None]
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, np.sum(dy * r * rstd[:, None], axis=0)


def _sigma(g):
    """The logistic function without overflow on either side."""
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def swiglu(gate, up):
    g, u = np.asarray(gate, np.float64), np.asarray(up, np.float64)
    return g * _sigma(g) * u


def swiglu_backward(dh, gate, up):
    dh, g, u = (np.asarray(t, np.float64) for t in (dh, gate, up))
    s = _sigma(g)
    return dh * u * (s + g * s * _sigma(-g)), dh * g * s


def grad_norm(grads):
    return np.sqrt(sum(np.sum(np.square(np.asarray(g, np.float64))) for g in grads))


def clip_factor(norm, max_norm):
    return max_norm / norm if norm > max_norm else 1.0


def code_errors(codes, scales, y, err, group, pow2):
    """How codes and scales [rows][cols / group] of a result differ from what a
    computation within `err` of the exact y [rows][cols] can give: (number of
    scales, number of codes out of reach).

    A float32 scale is amax/448 of values within err, and off by one rounding;
    a power-of-two byte is that of an amax in the same range.  A code is that of
    (y +- err) times 448/amax, off by the rounding of the factor and of the
    product (2^-24 each), and encoding is monotone."""
    rows, cols = y.shape
    y = np.asarray(y, np.float64).reshape(rows, cols // group, group)
    err = np.broadcast_to(np.asarray(err, np.float64), (rows, cols)).reshape(y.shape)
    codes = np.asarray(codes).reshape(y.shape)
    low = np.max(np.abs(y) - err, axis=2).clip(min=0)
    high = np.max(np.abs(y) + err, axis=2)
    if pow2:
        # (an amax of zero has e = 0, and one that may be zero any e down to the least)
        least = lambda a: np.ceil(np.log2(np.maximum(a, 1e-300) / E4M3_MAX)).clip(min=-127)
        e = np.asarray(scales, np.int64) - 127
        bad_scales = (e < least(low)) | ((e > least(high)) & ~((low == 0) & (e == 0)))
        s = np.exp2(e.astype(np.float64))
    else:
        s = np.asarray(scales, np.float64)
        unit = s == 1.0  # a group of zeros
        bad_scales = ((s < low / E4M3_MAX * (1 - 2 ** -23)) | (s > high / E4M3_MAX * (1 + 2 ** -23))) \
            & ~(unit & (low < 2.0 ** -117))
    v = y / s[..., None]
    reach = err / s[..., None] + np.abs(v) * 4 * 2.0 ** -24
    clip = lambda a: np.clip(a, -E4M3_MAX, E4M3_MAX).astype(np.float32)
    value = e4m3_decode(codes)
    # (float32 of the borders: one more rounding, in reach's favour)
    bad = (value < e4m3_decode(e4m3_encode(clip(v - reach)))) | \
          (value > e4m3_decode(e4m3_encode(clip(v + reach)))) | np.isnan(value)
    return int(bad_scales.sum()), int(bad.sum())
