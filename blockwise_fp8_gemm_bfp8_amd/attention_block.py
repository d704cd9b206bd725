"""A decoder layer's attention block, forward and backward, on preallocated
buffers: the FP8 QKV projection, rotary positions, causal attention over packed
sequences, and the FP8 output projection.

  forward:   x -> quantise -> QKV GEMM -> turn q and k in place -> attention
             -> quantise -> output GEMM -> y
  backward:  dy -> quantise -> output dgrad and wgrad -> attention's gradient,
             written as rows [dq | dk | dv] -> turn dq and dk back in place
             -> quantise -> QKV dgrad and wgrad -> dx, dw_qkv, dw_o

The linears run as in ``hotpath`` (Puro-2B paper translation, section 3.2: 1x128
groups and 128x128 weight blocks, both layouts of an activation from one read,
scales K-block major); attention and the rotation stay in bf16 (Puro-2B
tutorial, FP8/MuonH section).  q, k and v are never copied apart: attention
reads and writes the heads of the fused rows where they lie.  A pass only
enqueues kernels on the current stream, so it can be captured into a graph.
"""

import torch

from . import (attention_backward, attention_forward, attention_workspace_bytes, gemm,
               gemm_workspace_bytes, quantize_act_dual_kmajor, quantize_weight_batch, rope)


class AttentionBlock:
    """w_qkv [(heads + 2 kv_heads) head_dim][hidden], w_o [hidden][heads head_dim]
    (bfloat16, rows q heads, k heads, v heads); `tokens` rows a pass, in
    sequences starting at `cu` (int32 [batch+1], device); `table` from
    rope_table, `positions` int32 [tokens].  All sizes multiples of 128.

    The sequences need not fill the rows, and `cu` and `positions` may hold
    other values in every pass: rows of no sequence (before cu[0], from cu[-1]
    on) count as zeros where attention leaves off, so y and dx are 0 there and
    the weights' gradients take nothing from them, whatever their positions.
    x and dy must be finite there, as they share a 128-token group's scale.
    (BFP8_DEBUG's scan takes a position outside the table for what it gives: NaN.)"""

    def __init__(self, w_qkv, w_o, heads: int, kv_heads: int, tokens: int, cu, positions, table,
                 scale: float = None):
        rows, hidden = w_qkv.shape
        if rows % (heads + 2 * kv_heads):
            raise ValueError(f"w_qkv has {rows} rows, not a multiple of {heads + 2 * kv_heads} heads")
        D = rows // (heads + 2 * kv_heads)
        if tuple(w_o.shape) != (hidden, heads * D):
            raise ValueError(f"w_o must be [{hidden}][{heads * D}], got {tuple(w_o.shape)}")
        for name, n in (("tokens", tokens), ("hidden", hidden), ("w_qkv rows", rows),
                        ("heads * head_dim", heads * D)):
            if n % 128:
                raise ValueError(f"{name} must be a multiple of 128, got {n}")
        self.w_qkv, self.w_o = w_qkv, w_o
        self.heads, self.kv_heads, self.head_dim, self.scale = heads, kv_heads, D, scale
        self.cu, self.positions, self.table = cu, positions, table
        self._quantized = self._ran = False  # what the buffers hold
        dev, M, E = w_qkv.device, tokens, heads * D
        u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)

        def operand(name, cols):  # both layouts' codes and scales of an [M][cols] activation
            return {name + "q": new((M, cols), u8), name + "s": new((cols // 128, M), f32),
                    name + "qt": new((cols, M), u8), name + "st": new((M // 128, cols), f32)}

        b = self.buf = {}
        for name, w in (("wqkv", w_qkv), ("wo", w_o)):
            b[name + "_q"] = new(tuple(w.shape), u8)
            b[name + "_s"] = new((w.shape[0] // 128, w.shape[1] // 128), f32)
        for name, cols in (("x", hidden), ("a", E), ("dy", hidden), ("dqkv", rows)):
            b.update(operand(name, cols))
        b["qkv"], b["dqkv"] = new((M, heads + 2 * kv_heads, D), bf), new((M, heads + 2 * kv_heads, D), bf)
        b["a"], b["da"] = new((M, heads, D), bf), new((M, heads, D), bf)
        b["lse"] = new((heads, M), f32)
        b["y"], b["dx"] = new((M, hidden), bf), new((M, hidden), bf)
        b["dw_qkv"], b["dw_o"] = new((rows, hidden), bf), new((hidden, E), bf)
        need = max(gemm_workspace_bytes("NT", "act_km", "act_km", rows, hidden, M),
                   gemm_workspace_bytes("NT", "act_km", "act_km", hidden, E, M), 16)
        b["gemm_ws"] = new((need,), u8)
        q, k, v = self._heads(b["qkv"])
        need = max(attention_workspace_bytes(q, k, v, cu, cu, backward=back) for back in (False, True))
        b["attn_ws"] = new((max(need, 16),), u8)

    def _heads(self, rows):
        H, KV = self.heads, self.kv_heads
        return rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]

    def _check_rows(self, t, name):
        """The quantisers take their sizes from t and write to this block's buffers."""
        y = self.buf["y"]
        if t.shape != y.shape or t.device != y.device:
            raise ValueError(f"{name} must be {list(y.shape)} on {y.device}, got {list(t.shape)} on "
                             f"{t.device}")

    def _turn(self, rows, inverse):
        turned = rows[:, :self.heads + self.kv_heads]
        rope(turned, self.table, self.positions, inverse=inverse, out=turned)

    def quantize_weights(self):
        """Codes of both weights, once per optimizer step (and before the first forward)."""
        b = self.buf
        quantize_weight_batch([self.w_qkv, self.w_o], [b["wqkv_q"], b["wo_q"]],
                              [b["wqkv_s"], b["wo_s"]])
        self._quantized = True

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """y [tokens][hidden] of x [tokens][hidden] (bfloat16); the buffers keep
        what backward needs."""
        self._check_rows(x, "x")
        if not self._quantized:
            raise RuntimeError("quantize_weights() comes before the first forward")
        b = self.buf
        M = b["y"].shape[0]
        quantize_act_dual_kmajor(x, b["xq"], b["xs"], b["xqt"], b["xst"])
        gemm("NT", b["xq"], b["xs"], b["wqkv_q"], b["wqkv_s"], "act_km", "block",
             out=b["qkv"].view(M, -1), workspace=b["gemm_ws"])
        self._turn(b["qkv"], False)
        attention_forward(*self._heads(b["qkv"]), self.cu, self.cu, scale=self.scale, out=b["a"],
                          lse=b["lse"], workspace=b["attn_ws"], zero_rest=True)
        quantize_act_dual_kmajor(b["a"].view(M, -1), b["aq"], b["as"], b["aqt"], b["ast"])
        self._ran = True
        return gemm("NT", b["aq"], b["as"], b["wo_q"], b["wo_s"], "act_km", "block", out=b["y"],
                    workspace=b["gemm_ws"])

    def backward(self, dy: torch.Tensor):
        """(dx, dw_qkv, dw_o) for the gradient dy of the last forward's y."""
        self._check_rows(dy, "dy")
        if not self._ran:
            raise RuntimeError("forward() comes before backward")
        b = self.buf
        M = b["y"].shape[0]
        quantize_act_dual_kmajor(dy, b["dyq"], b["dys"], b["dyqt"], b["dyst"])
        gemm("NN", b["dyq"], b["dys"], b["wo_q"], b["wo_s"], "act_km", "block",
             out=b["da"].view(M, -1), workspace=b["gemm_ws"])
        gemm("NT", b["dyqt"], b["dyst"], b["aqt"], b["ast"], "act_km", "act_km", out=b["dw_o"],
             workspace=b["gemm_ws"])
        dq, dk, dv = self._heads(b["dqkv"])
        attention_backward(b["da"], *self._heads(b["qkv"]), b["a"], b["lse"], self.cu, self.cu,
                           scale=self.scale, dq=dq, dk=dk, dv=dv, workspace=b["attn_ws"],
                           zero_rest=True)
        self._turn(b["dqkv"], True)
        quantize_act_dual_kmajor(b["dqkv"].view(M, -1), b["dqkvq"], b["dqkvs"], b["dqkvqt"],
                                 b["dqkvst"])
        gemm("NN", b["dqkvq"], b["dqkvs"], b["wqkv_q"], b["wqkv_s"], "act_km", "block",
             out=b["dx"], workspace=b["gemm_ws"])
        gemm("NT", b["dqkvqt"], b["dqkvst"], b["xqt"], b["xst"], "act_km", "act_km",
             out=b["dw_qkv"], workspace=b["gemm_ws"])
        return b["dx"], b["dw_qkv"], b["dw_o"]
