"""What the tests of the layer operators share: inputs in padded rows, values as
float64, and the check of codes against an exact result."""
import numpy as np
import torch

from oracle import layer

U = 2.0 ** -24   # half a step of float32
EPS = 1e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # relative rounding of an output


def padded(rows, cols, dtype, gen, scale=1.0, extra=0):
    """[rows][cols] in rows that start 16-byte aligned, `extra` vectors apart;
    what lies between holds 777."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = -(-cols // per) * per + extra * per
    t = torch.full((max(rows, 1), ld), 777.0, dtype=dtype, device="cuda")
    t[:rows, :cols] = (torch.randn((rows, cols), device="cuda", generator=gen) * scale).to(dtype)
    return t[:rows, :cols]


def f64(t):
    return t.double().cpu().numpy()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def close(got, want, err, dtype=None):
    """got within err of want, and within one rounding to dtype beside it."""
    got, want = f64(got), np.asarray(want)
    rounding = HALF[dtype] * (np.abs(want) + err) if dtype is not None else 0.0
    worst = np.max(np.abs(got - want) / (err + rounding + 1e-38)) if got.size else 0.0
    assert np.all(np.isfinite(got)) and worst <= 1.0, worst


def check_codes(out, y, err, scales):
    """(q, s) or (q, s, qt, st) against the exact result y, computed within err."""
    group, pow2 = (32 if scales == "mx32" else 128), scales != "fp32"
    err = np.broadcast_to(err, y.shape)
    for k, (z, e) in enumerate([(y, err), (y.T, err.T)][:len(out) // 2]):
        q, s = out[2 * k].cpu().numpy(), out[2 * k + 1].cpu().numpy()
        assert q.shape == z.shape
        assert layer.code_errors(q, s if scales == "mx32" else s.T, z, e, group, pow2) == (0, 0), k


def as_quantised(bfp8, y, scales, transposed):
    """The codes that the package's quantisers make of y (float32)."""
    rows, cols = y.shape
    if not transposed:
        if scales == "fp32":
            return bfp8.quantize_act_kmajor(y)
        q, s = bfp8.quantize_mx_act(y, 32 if scales == "mx32" else 128)
        return q, s if scales == "mx32" else s.t()
    if scales == "fp32":
        return bfp8.quantize_act_dual_kmajor(y)
    return bfp8.quantize_mx_act_dual(y, 32) if scales == "mx32" else bfp8.quantize_mx_act_dual_kmajor(y)
