"""Cases and plain forms of what a decoder layer's training pass computes around
its linear layers: the RMS norm with the residual's addition, the gated
activation between gate/up and down, both with E4M3 codes of their results, the
gradients of both, and the gradients' global norm and clipping.

``run`` computes them with elementary torch operations in float32, or, with
``own`` set, through the package's entry points.
"""

import math

import torch

own = False

EPS = 1e-6
MAX_NORM = 1.0
MOST = 16384 * 6144  # values of a gate in the largest activation cases


# ---- cases ------------------------------------------------------------------

def _rows(name, op, rows, cols, dtype, codes, extra):
    """``codes``: "none", "rows" (groups along channels) or "both" (those, and
    groups of 128 tokens, transposed); ``extra``: with a residual (its gradient)."""
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "codes": codes,
            "extra": extra}


def _clip(name, sizes, dtype):
    return {"name": name, "op": "clip", "sizes": sizes, "dtype": dtype}


# weight gradients of one layer, hidden size 2048, 16 + 8 + 8 heads of 128, feed-forward 6144:
# QKV, output, gate/up and down projections and two norms
_LAYER = "8388608 4194304 25165824 12582912 2048 2048"


def listed():
    return [
        # one new token of each of 16 requests: the norm before a linear in a generation step
        _rows("norm_token", "norm", 16, 2048, "bf16", "rows", True),
        # the norm before a layer's QKV or gate/up projection in training, 4 sequences of 4096
        _rows("norm_layer", "norm", 16384, 2048, "bf16", "both", True),
        # a norm whose result stays as it is, float32, an odd width and an odd number of rows
        _rows("norm_odd", "norm", 5003, 1111, "f32", "none", False),
        # the gradient of the training norm, the residual's gradient added
        _rows("norm_grad_layer", "norm_grad", 16384, 2048, "bf16", "none", True),
        # the gradient at an odd size in float32
        _rows("norm_grad_odd", "norm_grad", 777, 1003, "f32", "none", False),
        # a generation step's activation between gate/up and down
        _rows("glu_token", "glu", 16, 6144, "bf16", "rows", False),
        # the same in training: codes for down's forward and weight gradient
        _rows("glu_layer", "glu", 16384, 6144, "bf16", "both", False),
        # its gradient in training: codes for gate/up's input and weight gradients
        _rows("glu_grad_layer", "glu_grad", 16384, 6144, "bf16", "both", False),
        # its gradient without codes, ragged
        _rows("glu_grad_odd", "glu_grad", 1999, 4100, "bf16", "none", False),
        # a model of a few small tensors: latency
        _clip("clip_small", "1 4097 77 2048 12345 640 9", "f32"),
        # one layer's gradients in bf16
        _clip("clip_layer", _LAYER, "bf16"),
        # two layers' gradients kept in float32
        _clip("clip_main", _LAYER + " " + _LAYER, "f32"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "glu", "glu_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        most = 8000000 if dtype == "bf16" else 4000000
        sizes = [_log_int(rng, 1, most) for _ in range(rng.randint(1, 40))]
        return _clip("", " ".join(str(n) for n in sizes), dtype)
    codes = "none" if op == "norm_grad" else rng.choice(["none", "rows", "both"])
    # (over one channel the norm's gradient is nothing but what cancelling leaves)
    cols = _log_int(rng, 8 if op == "norm_grad" else 1, 16384)
    if codes != "none":
        cols = 128 * _log_int(rng, 1, 128)
    most = MOST // (8 if dtype == "f32" else 4)
    rows = _log_int(rng, 1, max(1, min(32768, most // cols)))
    if codes == "both":
        rows = 128 * _log_int(rng, 1, max(1, min(256, most // cols // 128)))
    return _rows("", op, rows, cols, dtype, codes,
                 op in ("norm", "norm_grad") and rng.random() < 0.7)


# ---- inputs -----------------------------------------------------------------

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _sizes(case):
    return [int(n) for n in case["sizes"].split()]


def _normal(rows, cols, scale, gen, dtype):
    """Rows as the framework keeps them: every one starts 16-byte aligned."""
    width = -(-cols // 8) * 8
    return (torch.randn((rows, width), device="cuda", generator=gen) * scale).to(dtype)[:, :cols]


def _prepare_rows(case, gen):
    rows, cols, dtype = case["rows"], case["cols"], _DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        # a residual stream: some channels far larger than the rest
        x = _normal(rows, cols, 1.0, gen, dtype)
        x[:, 5::199] *= 20
        state["w"] = 1.0 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
        if case["op"] == "norm":
            state["x"] = x
            state["residual"] = _normal(rows, cols, 2.0, gen, dtype) if case["extra"] else None
            return state
        state["r"] = x
        state["rstd"] = torch.rsqrt(x.double().square().mean(1) + EPS).float()
        state["dy"] = _normal(rows, cols, 1e-3, gen, dtype)
        state["dsum"] = _normal(rows, cols, 1e-3, gen, dtype) if case["extra"] else None
        return state
    # gate and up side by side in the rows of their one projection
    width = -(-cols // 8) * 8
    gate_up = _normal(rows, 2 * width, 1.5, gen, dtype)
    state["gate"], state["up"] = gate_up[:, :cols], gate_up[:, width:width + cols]
    if case["op"] == "glu_grad":
        state["dh"] = _normal(rows, cols, 1e-3, gen, dtype)
    return state


def _prepare_clip(case, gen):
    sizes, dtype = _sizes(case), _DTYPES[case["dtype"]]
    # tensors of one model differ in size of gradient; their norm lies over the limit
    total = sum(sizes)
    grads = [(torch.randn(n, device="cuda", generator=gen) *
              (4.0 * (0.5 + i % 4) / math.sqrt(total))).to(dtype) for i, n in enumerate(sizes)]
    state = {"case": case, "grads": grads}
    if own:
        import blockwise_fp8_gemm_bfp8_amd as bfp8

        state["plan"] = bfp8.GradClip(grads, [torch.empty_like(g) for g in grads])
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_clip(case, gen) if case["op"] == "clip" else _prepare_rows(case, gen)


# ---- plain forms ------------------------------------------------------------

def _scale(amax):
    """A group's float32 scale and the factor of its elements."""
    one = torch.ones_like(amax)
    return torch.where(amax == 0, one, amax / 448), torch.where(amax == 0, one, 448 / amax)


def _code(y):
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


def _codes(y, codes):
    """E4M3 codes of y [rows][cols] in groups of 128 channels, scales
    [cols/128][rows], and ("both") of its transpose in groups of 128 tokens,
    scales [rows/128][cols]."""
    rows, cols = y.shape
    groups = y.view(rows, cols // 128, 128)
    s, inv = _scale(groups.abs().amax(2))
    out = [_code(groups * inv[..., None]).view(rows, cols), s.t().contiguous()]
    if codes == "both":
        groups = y.view(rows // 128, 128, cols)
        s, inv = _scale(groups.abs().amax(1))
        out += [_code((groups * inv[:, None]).view(rows, cols).t().contiguous()), s]
    return out


def _plain_norm(state):
    case, x = state["case"], state["x"]
    r = x
    if state["residual"] is not None:
        r = (x.float() + state["residual"].float()).to(x.dtype)
    f = r.float()
    rstd = torch.rsqrt((f * f).mean(1) + EPS)
    y = f * rstd[:, None] * state["w"]
    out = [y.to(x.dtype)] if case["codes"] == "none" else _codes(y, case["codes"])
    return out + ([r] if case["extra"] else []) + [rstd]


def _plain_norm_grad(state):
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xh = state["r"].float() * rstd
    g = dy * state["w"]
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if state["dsum"] is not None:
        dx = dx + state["dsum"].float()
    return [dx.to(state["dy"].dtype), (dy * xh).sum(0)]


def _plain_glu(state):
    case, g = state["case"], state["gate"].float()
    h = g / (1 + (-g).exp()) * state["up"].float()
    return [h.to(state["gate"].dtype)] if case["codes"] == "none" else _codes(h, case["codes"])


def _plain_glu_grad(state):
    case, dtype = state["case"], state["gate"].dtype
    g, u, dh = state["gate"].float(), state["up"].float(), state["dh"].float()
    sig = 1 / (1 + (-g).exp())
    dgate, dup = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    if case["codes"] == "none":
        return [dgate.to(dtype), dup.to(dtype)]
    return _codes(torch.cat([dgate, dup], 1), case["codes"])


def _plain_clip(state):
    grads = state["grads"]
    norm = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
    c = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm))
    return [(g.float() * c).to(g.dtype) for g in grads] + [norm]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "glu": _plain_glu,
                "glu_grad": _plain_glu_grad, "clip": _plain_clip}[op](state)
    import blockwise_fp8_gemm_bfp8_amd as bfp8

    if op == "clip":
        norm = state["plan"].clip(MAX_NORM)
        return state["plan"].out + [norm]
    if op == "norm_grad":
        return list(bfp8.rmsnorm_backward(state["dy"], state["r"], state["w"], state["rstd"],
                                          state["dsum"]))
    both = case["codes"] == "both"
    if op == "norm":
        if case["codes"] == "none":
            y, r, rstd = bfp8.rmsnorm(state["x"], state["w"], state["residual"], eps=EPS)
            out = [y]
        else:
            *out, r, rstd = bfp8.rmsnorm_quantize(state["x"], state["w"], state["residual"],
                                                  eps=EPS, transposed=both)
        return _as_values(out) + ([r] if case["extra"] else []) + [rstd]
    if op == "glu":
        if case["codes"] == "none":
            return [bfp8.swiglu(state["gate"], state["up"])]
        return _as_values(bfp8.swiglu_quantize(state["gate"], state["up"], transposed=both))
    if case["codes"] == "none":
        return list(bfp8.swiglu_backward(state["dh"], state["gate"], state["up"]))
    return _as_values(bfp8.swiglu_backward_quantize(state["dh"], state["gate"], state["up"],
                                                    transposed=both))


def _as_values(out):
    """Codes are returned as the E4M3 values they are."""
    return [t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for t in out]


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * size + 4, "flops": 3 * n}
    rows, cols, op = case["rows"], case["cols"], case["op"]
    n, weight, per_row = rows * cols, 4 * cols, 4 * rows
    outputs = 2 if op == "glu_grad" else 1
    if case["codes"] == "none":
        written = size * n * outputs
    else:
        kinds = 2 if case["codes"] == "both" else 1
        written = kinds * outputs * (n + 4 * n // 128)
    if op == "norm":  # x, residual and their sum, the weight, the rows' statistics
        return {"bytes": n * size * (3 if case["extra"] else 1) + written + weight + per_row,
                "flops": 5 * n}
    if op == "norm_grad":
        return {"bytes": n * size * (3 if case["extra"] else 2) + written + 2 * weight + per_row,
                "flops": 10 * n}
    return {"bytes": n * size * (3 if op == "glu_grad" else 2) + written,
            "flops": (12 if op == "glu_grad" else 5) * n}


# ---- 64-bit values ----------------------------------------------------------

def _exact_codes(y, codes):
    """Scaled values before their rounding to E4M3, and the scales."""
    rows, cols = y.shape
    out = []
    for z in ([y] if codes == "rows" else [y, y.t()]):
        # [groups][other axis][128]
        blocks = torch.stack(z.split(128, 1))
        scale = blocks.abs().amax(2) / 448
        scale[scale == 0] = 1
        out += [torch.cat(list(blocks / scale[..., None]), 1), scale]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        grads = [g.double() for g in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(g, g)) for g in grads))
        return [g * min(1.0, MAX_NORM / norm) for g in grads] + [torch.tensor(norm, dtype=torch.float64)]
    if case["op"] == "norm":
        r = s["x"].double()
        if s["residual"] is not None:  # the stream is kept in the tensors' type, and the norm is of that
            r = (r + s["residual"].double()).to(s["x"].dtype).double()
        rstd = (r.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        y = torch.einsum("tc,t,c->tc", r, rstd, s["w"].double())
        out = [y] if case["codes"] == "none" else _exact_codes(y, case["codes"])
        return out + ([r] if case["extra"] else []) + [rstd]
    if case["op"] == "norm_grad":
        r, dy, w, rstd = s["r"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
        dot = (dy * w * r).sum(1)
        dx = dy * w * rstd[:, None] - r * (dot * rstd.pow(3) / case["cols"])[:, None]
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return [dx, torch.einsum("tc,tc,t->c", dy, r, rstd)]
    g, u = s["gate"].double(), s["up"].double()
    if case["op"] == "glu":
        h = g * torch.sigmoid(g) * u
        return [h] if case["codes"] == "none" else _exact_codes(h, case["codes"])
    dh, sig = s["dh"].double(), torch.sigmoid(g)
    dgate, dup = dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * sig * g
    if case["codes"] == "none":
        return [dgate, dup]
    return _exact_codes(torch.cat([dgate, dup], 1), case["codes"])
