"""Cases and plain forms of the operators between a decoder layer's QKV and
output projections: rotary positions, attention and attention's gradient.

``run`` computes them with elementary torch operations in float32, or, with
``own`` set, through the package's entry points.
"""

import math

import torch

own = False

MAX_PAIRS = 16 * 16384 * 16385 // 2 * 128  # visible pairs x q heads x head size of the largest case


# ---- cases ------------------------------------------------------------------

def _rope(name, tokens, heads, row_heads, dim, rot, layout, scaling, inverse, dtype, length, order):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "row_heads": row_heads,
            "dim": dim, "rot": rot, "layout": layout, "scaling": scaling, "inverse": inverse,
            "dtype": dtype, "length": length, "order": order}


def _attn(name, op, heads, kv_heads, dim, causal, layout, q_lens, k_lens, k_rows=0):
    return {"name": name, "op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": causal, "layout": layout, "q_lens": q_lens, "k_lens": k_lens,
            "k_rows": k_rows}


def _text(lens):
    return " ".join(str(n) for n in lens)


def _lens(text):
    return [int(n) for n in text.split()]


# Documents packed into one micro-batch of 2 x 4096 tokens, as a pretraining loader packs them.
_DOCS = "1 2417 64 913 127 129 1500 333 17 2000 8 255 428"
# Cached lengths of 16 requests under way, each with room for 4096 tokens.
_CACHED = "4096 1 37 4095 2048 777 3333 128 129 1024 64 3999 512 2500 63 1801"


def listed():
    layer = _text([4096] * 4)
    return [
        # the q and k heads of a layer's fused QKV rows, 4 sequences of 4096
        _rope("rope_layer", 16384, 24, 32, 128, 128, "half", "none", False, "bf16", 4096, "packed"),
        # one new token of each of 16 requests: what a generation step pays
        _rope("rope_token", 16, 24, 32, 128, 128, "half", "linear", False, "bf16", 8192, "spread"),
        # the gradient, interleaved pairs over part of each head, contexts stretched by YaRN, an odd count
        _rope("rope_partial_grad", 5003, 12, 12, 96, 64, "interleaved", "yarn", True, "f32", 16384,
              "spread"),
        # a layer's attention in training: 4 sequences of 4096
        _attn("forward_layer", "forward", 16, 8, 128, True, "fused", layer, layer),
        # one long sequence
        _attn("forward_long", "forward", 16, 8, 128, True, "fused", "16384", "16384"),
        # a micro-batch of packed documents of ragged lengths
        _attn("forward_packed", "forward", 16, 8, 128, True, "fused", _DOCS, _DOCS),
        # short queries over longer memories, no causal mask, plain heads of 64 stored head by head
        _attn("forward_cross", "forward", 8, 8, 64, False, "heads", "129 200", "333 77"),
        # generation: one query a request over its cache
        _attn("forward_token", "forward", 16, 8, 128, True, "cache", _text([1] * 16), _CACHED, 4096),
        # the gradients of the same
        _attn("backward_layer", "backward", 16, 8, 128, True, "fused", layer, layer),
        _attn("backward_long", "backward", 16, 8, 128, True, "fused", "16384", "16384"),
        _attn("backward_packed", "backward", 16, 8, 128, True, "fused", _DOCS, _DOCS),
        _attn("backward_cross", "backward", 8, 8, 64, False, "heads", "129 200", "333 77"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if work(case)["flops"] <= 10 * MAX_PAIRS:  # no more than the largest listed case
            return case


def _draw(rng):
    kind = rng.choice(["rope", "forward", "forward", "backward", "backward", "token"])
    if kind == "rope":
        dim = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        heads = rng.randint(1, 40)
        tokens = _log_int(rng, 1, min(32768, 16384 * 24 * 128 // (heads * dim)))
        return _rope("", tokens, heads, heads + rng.choice([0, 0, 1, 8]), dim, rot,
                     rng.choice(["half", "interleaved"]),
                     rng.choice(["none", "linear", "ntk", "yarn"]), rng.random() < 0.5,
                     rng.choice(["bf16", "bf16", "f32"]), rng.choice([2048, 4096, 16384, 65536]),
                     rng.choice(["packed", "spread"]))
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4])
    dim = rng.choice([32, 64, 64, 80, 128, 128, 128])
    if kind == "token":
        rows = _log_int(rng, 16, 16384)
        batch = _log_int(rng, 1, min(64, max(1, 262144 // rows)))
        lens = [_log_int(rng, 1, rows) for _ in range(batch)]
        queries = [rng.choice([1, 1, 1, 2, 5]) for _ in range(batch)]
        queries = [min(a, b) for a, b in zip(queries, lens)]
        return _attn("", "forward", heads, kv_heads, dim, True, "cache", _text(queries),
                     _text(lens), rows)
    total = _log_int(rng, 16, 16384)
    count = _log_int(rng, 1, min(64, total))
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    q_lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    layout = rng.choice(["fused", "fused", "heads"])
    causal = rng.random() < 0.75
    k_lens = q_lens
    if layout == "heads":
        k_lens = [n + rng.randint(0, 300) if causal else _log_int(rng, 1, 2048) for n in q_lens]
    return _attn("", kind, heads, kv_heads, dim, causal, layout, _text(q_lens), _text(k_lens))


# ---- inputs -----------------------------------------------------------------

def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _normal(shape, scale, gen, dtype):
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)


_SCALING = {"none": (1.0, 0), "linear": (2.0, 0), "ntk": (4.0, 0), "yarn": (4.0, 4096)}


def _prepare_rope(case, gen):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]]
    T, H, D, length = case["tokens"], case["heads"], case["dim"], case["length"]
    rows = _normal((T, case["row_heads"], D), 1.0, gen, dtype)
    if case["order"] == "packed":
        positions = torch.arange(T, device="cuda", dtype=torch.int32) % length
    else:
        positions = torch.randint(0, length, (T,), device="cuda", generator=gen, dtype=torch.int32)
    factor, original = _SCALING[case["scaling"]]
    state = {"case": case, "x": rows[:, :H], "positions": positions}
    if own:
        import blockwise_fp8_gemm_bfp8_amd as bfp8

        state["table"] = bfp8.rope_table(length, case["rot"], base=10000.0, scaling=case["scaling"],
                                         factor=factor, original_length=original, device="cuda")
    else:
        state["table"] = _plain_table(length, case["rot"], case["scaling"], factor, original)
    return state


def _plain_table(length, rot, scaling, factor, original):
    """[length][rot / 2][cos, sin], angles taken in 64 bits (a product of a
    position and a frequency in 32 would be off by 1e-3 at 16384)."""
    base = 10000.0
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    magnitude = 1.0
    if scaling == "linear":
        freq = freq / factor
    if scaling == "yarn":
        turns = original * freq / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        magnitude = 0.1 * math.log(factor) + 1
    angle = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * freq
    return (torch.stack([angle.cos(), angle.sin()], -1) * magnitude).float()


def _prepare_attention(case, gen):
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    Tq, rows = sum(q_lens), case["k_rows"]
    Tk = rows * len(k_lens) if rows else sum(k_lens)
    bf = torch.bfloat16
    if case["layout"] == "fused":  # q, k and v heads side by side in the QKV projection's rows
        qkv = _normal((Tq, H + 2 * KV, D), 1.0, gen, bf)
        q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    elif case["layout"] == "heads":  # every head's tokens in a row of their own
        q = _normal((H, Tq, D), 1.0, gen, bf).transpose(0, 1)
        k = _normal((KV, Tk, D), 1.0, gen, bf).transpose(0, 1)
        v = _normal((KV, Tk, D), 1.0, gen, bf).transpose(0, 1)
    else:  # a cache of `k_rows` rows a request, its k and v apart
        q = _normal((Tq, H, D), 1.0, gen, bf)
        k = _normal((Tk, KV, D), 1.0, gen, bf)
        v = _normal((Tk, KV, D), 1.0, gen, bf)
    # some features of real activations are far larger than the rest
    q[..., 3::29] *= 2
    i32 = dict(dtype=torch.int32, device="cuda")
    state = {"case": case, "q": q, "k": k, "v": v, "q_lens": q_lens, "k_lens": k_lens,
             "scale": 1.0 / math.sqrt(D), "cu_q": torch.tensor(_starts(q_lens), **i32)}
    if rows:
        state["k_starts"] = [rows * b for b in range(len(k_lens))]
        state["cu_k"] = torch.tensor(_starts([rows] * len(k_lens)), **i32)
        state["used"] = torch.tensor(k_lens, **i32)
    else:
        state["k_starts"] = _starts(k_lens)[:-1]
        state["cu_k"] = torch.tensor(_starts(k_lens), **i32)
        state["used"] = None
    if case["op"] == "backward":  # what the forward pass left, and the gradient that arrives
        state["out"], state["lse"] = _plain_forward(state)
        state["dout"] = _normal((Tq, H, D), 1e-3, gen, bf)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_rope(case, gen) if case["op"] == "rope" else _prepare_attention(case, gen)


# ---- plain forms ------------------------------------------------------------

def _plain_rope(state):
    case, x = state["case"], state["x"].float()
    rot = case["rot"]
    table = state["table"][state["positions"].long()][:, None]
    c, s = table[..., 0], table[..., 1]
    if case["inverse"]:
        s = -s
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * c - b * s
        y[..., rot // 2:rot] = a * s + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * s
        y[..., 1:rot:2] = a * s + b * c
    return y.to(state["x"].dtype)


def _pieces(state):
    """(query rows, key rows, kv head, hidden pairs) of the plain forms: the
    heads of one kv head of one sequence at a time, so that the matrices of
    all pairs stay small."""
    case = state["case"]
    at = 0
    for n, m, k0 in zip(state["q_lens"], state["k_lens"], state["k_starts"]):
        hidden = None
        if case["causal"]:  # query i sees keys up to i + m - n
            i = torch.arange(n, device="cuda")[:, None]
            hidden = torch.arange(m, device="cuda")[None] > i + (m - n)
        if n:
            for g in range(case["kv_heads"]):
                yield slice(at, at + n), slice(k0, k0 + m), g, hidden
        at += n


def _scores(state, rows, keys, g, hidden):
    group = state["case"]["heads"] // state["case"]["kv_heads"]
    q = state["q"][rows, g * group:(g + 1) * group].float().transpose(0, 1)
    k = state["k"][keys, g].float()
    s = q @ k.t() * state["scale"]
    if hidden is not None:
        s = s.masked_fill(hidden, float("-inf"))
    return q, k, s


def _plain_forward(state):
    case, q = state["case"], state["q"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.full((case["heads"], q.shape[0]), float("-inf"), device="cuda")
    for rows, keys, g, hidden in _pieces(state):
        _, _, s = _scores(state, rows, keys, g, hidden)
        top = s.amax(-1, keepdim=True)
        p = (s - top).exp()
        total = p.sum(-1, keepdim=True)
        o = p @ state["v"][keys, g].float() / total
        heads = slice(g * group, (g + 1) * group)
        out[rows, heads] = o.transpose(0, 1).to(q.dtype)
        lse[heads, rows] = (total.log() + top)[..., 0]
    return out, lse


def _plain_backward(state):
    case = state["case"]
    group = case["heads"] // case["kv_heads"]
    dq, dk, dv = (torch.zeros(state[n].shape, dtype=state[n].dtype, device="cuda") for n in "qkv")
    for rows, keys, g, hidden in _pieces(state):
        heads = slice(g * group, (g + 1) * group)
        q, k, s = _scores(state, rows, keys, g, hidden)
        p = (s - state["lse"][heads, rows][..., None]).exp()
        v = state["v"][keys, g].float()
        do = state["dout"][rows, heads].float().transpose(0, 1)
        delta = (do * state["out"][rows, heads].float().transpose(0, 1)).sum(-1, keepdim=True)
        ds = p * (do @ v.t() - delta) * state["scale"]
        dq[rows, heads] = (ds @ k).transpose(0, 1).to(dq.dtype)
        # the gradient of a shared head is the sum over the q heads that read it
        dk[keys, g] = (ds.flatten(0, 1).t() @ q.flatten(0, 1)).to(dk.dtype)
        dv[keys, g] = (p.flatten(0, 1).t() @ do.flatten(0, 1)).to(dv.dtype)
    return dq, dk, dv


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "rope":
            return _plain_rope(state)
        return _plain_forward(state) if case["op"] == "forward" else _plain_backward(state)
    import blockwise_fp8_gemm_bfp8_amd as bfp8

    if case["op"] == "rope":
        return bfp8.rope(state["x"], state["table"], state["positions"], layout=case["layout"],
                         inverse=case["inverse"])
    shape = dict(cu_q=state["cu_q"], cu_k=state["cu_k"], k_lens=state["used"],
                 causal=case["causal"], scale=state["scale"])
    if case["op"] == "forward":
        return bfp8.attention_forward(state["q"], state["k"], state["v"], **shape)
    return bfp8.attention_backward(state["dout"], state["q"], state["k"], state["v"],
                                   state["out"], state["lse"], **shape)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        T, H, D, rot = case["tokens"], case["heads"], case["dim"], case["rot"]
        table = min(T, case["length"]) * rot * 4
        return {"bytes": 2 * T * H * D * size + 4 * T + table, "flops": 3 * T * H * rot}
    q_lens, k_lens = _lens(case["q_lens"]), _lens(case["k_lens"])
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    pairs = 0
    for n, m in zip(q_lens, k_lens):
        if not case["causal"]:
            pairs += n * m
        elif m >= n:
            pairs += n * (m - n) + n * (n + 1) // 2
        else:
            pairs += m * (m + 1) // 2
    q_bytes, kv_bytes, lse = 2 * sum(q_lens) * H * D, 2 * 2 * sum(k_lens) * KV * D, 4 * sum(q_lens) * H
    if case["op"] == "forward":
        return {"bytes": 2 * q_bytes + kv_bytes + lse, "flops": 4 * pairs * H * D}
    return {"bytes": 4 * q_bytes + 2 * kv_bytes + lse, "flops": 10 * pairs * H * D}


# ---- 64-bit values ----------------------------------------------------------

def _exact_rope(case, state):
    factor, original = _SCALING[case["scaling"]]
    rot, x = case["rot"], state["x"].double()
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base = 10000.0
    if case["scaling"] == "ntk" and rot > 2:
        base = base * math.pow(factor, rot / (rot - 2.0))
    f = torch.exp(-2.0 * i / rot * math.log(base))
    m = 1.0
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "yarn":
        ramp = torch.clamp((original * f / (2.0 * math.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = (1.0 - ramp) * f / factor + ramp * f
        m = 1.0 + 0.1 * math.log(factor)
    turn = state["positions"].double()[:, None, None] * f
    if case["inverse"]:
        turn = -turn
    first = torch.arange(rot // 2, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (rot // 2 if case["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(turn, m), turn)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_attention(case, state):
    """One q head of one sequence at a time, from softmax's definition and,
    for the gradients, from its derivative."""
    forward = case["op"] == "forward"
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(state["q"].shape, **f64), torch.full((H, state["q"].shape[0]),
                                                               float("-inf"), **f64)
    grads = [torch.zeros(state[n].shape, **f64) for n in "qkv"]
    r0 = 0
    for b, (n, m) in enumerate(zip(state["q_lens"], state["k_lens"])):
        r1, k0 = r0 + n, state["k_starts"][b]
        k1 = k0 + m
        for h in range(H if n and m else 0):
            g = h * KV // H
            q, k, v = state["q"][r0:r1, h].double(), state["k"][k0:k1, g].double(), \
                state["v"][k0:k1, g].double()
            a = (q @ k.t()) / math.sqrt(D)
            if case["causal"]:
                seen = torch.ones((n, m), dtype=torch.bool, device="cuda").tril_(m - n)
                a.masked_fill_(~seen, -math.inf)
            logz = torch.logsumexp(a, 1)
            w = torch.exp(a.sub_(logz.clamp(min=-1e300)[:, None]))
            out[r0:r1, h], lse[h, r0:r1] = w @ v, logz
            if not forward:
                do = state["dout"][r0:r1, h].double()
                dw = do @ v.t()
                da = w * (dw - (w * dw).sum(1, keepdim=True)) / math.sqrt(D)
                grads[0][r0:r1, h] = da @ k
                grads[1][k0:k1, g] += da.t() @ q
                grads[2][k0:k1, g] += w.t() @ do
        r0 = r1
    return (out, lse) if forward else tuple(grads)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, state)
    return _exact_attention(case, state)
