"""A decoder layer's feed-forward block, forward and backward, on preallocated
buffers: the residual's addition and the RMS norm, the FP8 gate/up projection,
the gated activation, and the FP8 down projection.

  forward:   x, residual -> r = x + residual, codes of norm(r) -> gate/up GEMM
             -> codes of silu(gate) up -> down GEMM -> y; r goes on
  backward:  dy -> quantise -> down dgrad and wgrad -> codes of [dgate | dup]
             -> gate/up dgrad and wgrad -> the norm's gradient, the gradient of
             r added -> dx (of x and of the residual), dw_gate_up, dw_down, dw_norm

The linears run as in ``hotpath`` (Puro-2B paper translation, section 3.2: 1x128
groups and 128x128 weight blocks, both layouts of an activation, scales K-block
major).  The normed rows, the activation and its gradient exist as codes only:
they go from registers to E4M3 in the kernels that compute them.  A pass only
enqueues kernels on the current stream, so it can be captured into a graph.
"""

import torch

from . import (gemm, gemm_workspace_bytes, quantize_act_dual_kmajor, quantize_weight_batch,
               rmsnorm_backward, rmsnorm_backward_workspace_bytes, rmsnorm_quantize,
               swiglu_backward_quantize, swiglu_quantize)


class MLPBlock:
    """w_norm [hidden] (bfloat16 or float32), w_gate_up [2 ffn][hidden] (gate rows,
    then up rows), w_down [hidden][ffn] (bfloat16); `tokens` rows a pass.  All sizes
    multiples of 128.

    A token group's scale is shared by 128 rows: rows that count for nothing must
    be finite, and zero in dy and dr for the weights' gradients to take nothing
    from them."""

    def __init__(self, w_norm, w_gate_up, w_down, tokens: int, eps: float = 1e-6):
        hidden, ffn = w_down.shape
        if tuple(w_gate_up.shape) != (2 * ffn, hidden):
            raise ValueError(f"w_gate_up must be [{2 * ffn}][{hidden}], got {tuple(w_gate_up.shape)}")
        if tuple(w_norm.shape) != (hidden,):
            raise ValueError(f"w_norm must be [{hidden}], got {tuple(w_norm.shape)}")
        for name, n in (("tokens", tokens), ("hidden", hidden), ("ffn", ffn)):
            if n % 128:
                raise ValueError(f"{name} must be a multiple of 128, got {n}")
        self.w_norm, self.w_gate_up, self.w_down, self.eps, self.ffn = w_norm, w_gate_up, w_down, eps, ffn
        self._quantized = self._ran = False  # what the buffers hold
        dev, M = w_down.device, tokens
        u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)

        def operand(cols):  # both layouts' codes and scales of an [M][cols] activation
            return {"q": new((M, cols), u8), "s": new((cols // 128, M), f32),
                    "qt": new((cols, M), u8), "st": new((M // 128, cols), f32)}

        self.x, self.h, self.dy, self.dgu = (operand(n) for n in (hidden, ffn, hidden, 2 * ffn))
        b = self.buf = {}
        for name, w in (("wgu", w_gate_up), ("wd", w_down)):
            b[name + "_q"] = new(tuple(w.shape), u8)
            b[name + "_s"] = new((w.shape[0] // 128, w.shape[1] // 128), f32)
        b["r"], b["rstd"] = new((M, hidden), bf), new((M,), f32)
        b["gate_up"], b["y"] = new((M, 2 * ffn), bf), new((M, hidden), bf)
        b["dh"], b["dn"], b["dx"] = new((M, ffn), bf), new((M, hidden), bf), new((M, hidden), bf)
        b["dw_gate_up"], b["dw_down"] = new((2 * ffn, hidden), bf), new((hidden, ffn), bf)
        b["dw_norm"] = new((hidden,), f32)
        gemms = [("NT", "act_km", "block", M, 2 * ffn, hidden), ("NT", "act_km", "block", M, hidden, ffn),
                 ("NN", "act_km", "block", M, ffn, hidden), ("NN", "act_km", "block", M, hidden, 2 * ffn),
                 ("NT", "act_km", "act_km", 2 * ffn, hidden, M), ("NT", "act_km", "act_km", hidden, ffn, M)]
        need = max(*(gemm_workspace_bytes(*g) for g in gemms),
                   rmsnorm_backward_workspace_bytes(M, hidden), 16)
        b["ws"] = new((need,), u8)

    def _check_rows(self, t, name):
        """The kernels take their sizes from t and write to this block's buffers."""
        y = self.buf["y"]
        if t.shape != y.shape or t.device != y.device or t.dtype != y.dtype:
            raise ValueError(f"{name} must be {y.dtype} {list(y.shape)} on {y.device}, got {t.dtype} "
                             f"{list(t.shape)} on {t.device}")
        if t.stride(1) != 1:  # dr is read last: not in mid-pass
            raise ValueError(f"{name} must have rows of unit stride, got strides {t.stride()}")

    def quantize_weights(self):
        """Codes of both weights, once per optimizer step (and before the first forward)."""
        b = self.buf
        quantize_weight_batch([self.w_gate_up, self.w_down], [b["wgu_q"], b["wd_q"]],
                              [b["wgu_s"], b["wd_s"]])
        self._quantized = True

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(y, r) for x and the residual stream [tokens][hidden] (bfloat16): r = x +
        residual is the stream that goes on, to which y is yet to be added.  The
        buffers keep what backward needs; y and r are two of them."""
        self._check_rows(x, "x")
        self._check_rows(residual, "residual")
        if not self._quantized:
            raise RuntimeError("quantize_weights() comes before the first forward")
        b, F = self.buf, self.ffn
        rmsnorm_quantize(x, self.w_norm, residual, eps=self.eps, transposed=True, **self.x,
                         sum_out=b["r"], rstd=b["rstd"])
        gemm("NT", self.x["q"], self.x["s"], b["wgu_q"], b["wgu_s"], "act_km", "block",
             out=b["gate_up"], workspace=b["ws"])
        swiglu_quantize(b["gate_up"][:, :F], b["gate_up"][:, F:], transposed=True, **self.h)
        gemm("NT", self.h["q"], self.h["s"], b["wd_q"], b["wd_s"], "act_km", "block", out=b["y"],
             workspace=b["ws"])
        self._ran = True
        return b["y"], b["r"]

    def backward(self, dy: torch.Tensor, dr: torch.Tensor):
        """(dx, dw_gate_up, dw_down, dw_norm) for the gradients dy of the last
        forward's y and dr of its r; dx is the gradient of x and of the residual."""
        self._check_rows(dy, "dy")
        self._check_rows(dr, "dr")
        if not self._ran:
            raise RuntimeError("forward() comes before backward")
        b, F = self.buf, self.ffn
        quantize_act_dual_kmajor(dy, **self.dy)
        gemm("NN", self.dy["q"], self.dy["s"], b["wd_q"], b["wd_s"], "act_km", "block", out=b["dh"],
             workspace=b["ws"])
        gemm("NT", self.dy["qt"], self.dy["st"], self.h["qt"], self.h["st"], "act_km", "act_km",
             out=b["dw_down"], workspace=b["ws"])
        swiglu_backward_quantize(b["dh"], b["gate_up"][:, :F], b["gate_up"][:, F:], transposed=True,
                                 **self.dgu)
        gemm("NN", self.dgu["q"], self.dgu["s"], b["wgu_q"], b["wgu_s"], "act_km", "block",
             out=b["dn"], workspace=b["ws"])
        gemm("NT", self.dgu["qt"], self.dgu["st"], self.x["qt"], self.x["st"], "act_km", "act_km",
             out=b["dw_gate_up"], workspace=b["ws"])
        rmsnorm_backward(b["dn"], b["r"], self.w_norm, b["rstd"], dr, dx=b["dx"],
                         dweight=b["dw_norm"], workspace=b["ws"])
        return b["dx"], b["dw_gate_up"], b["dw_down"], b["dw_norm"]
