"""Binding of include/bfp8_attention.h: rotary positions, attention and its
gradient on tensors of heads [tokens][heads][head_dim], whatever their strides
(the heads of a fused projection's rows, tensors stored head by head, caches).

Argument marshalling only, as in the package's other calls: every step runs in
the HIP kernels of libbfp8.so on the current stream of the tensors' device.
"""

import ctypes
import math

import torch

from . import DTYPES, AttentionShape, Heads, _check, _stream, lib

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _check_heads(t: torch.Tensor, name: str, dtypes, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens][heads][head_dim]")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.numel() and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last axis")


def _strides(t: torch.Tensor):
    """(row, head) strides; those of axes with one entry do not matter and
    take the values of a dense tensor."""
    T, H, D = t.shape
    head = t.stride(1) if H > 1 else D
    return (t.stride(0) if T > 1 else max(H * head, D)), head


def _heads(t: torch.Tensor) -> Heads:
    row, head = _strides(t)
    return Heads(t.data_ptr(), row, head)


def _check_i32(t, name: str, n: int, device):
    if t is None:
        return
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a dense 1-D int32 tensor on {device}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")


def _pointer(t):
    return None if t is None else t.data_ptr()


# ---- rotary positions -------------------------------------------------------

def rope_table(length: int, rot_dim: int, base: float = 10000.0, scaling: str = "none",
               factor: float = 1.0, original_length: int = 0, device="cuda",
               out: torch.Tensor = None) -> torch.Tensor:
    """float32 [length][rot_dim/2][2] cosines and sines of positions 0 ..
    length-1; `scaling` "none", "linear", "ntk" or "yarn" (see
    bfp8_rope_table)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    if out is None:
        if length < 0 or rot_dim < 0:
            raise ValueError("length and rot_dim must not be negative")
        out = torch.empty((length, rot_dim // 2, 2), dtype=torch.float32, device=device)
    elif (out.shape != (length, rot_dim // 2, 2) or out.dtype != torch.float32
          or not out.is_contiguous() or not out.is_cuda):
        raise ValueError("out must be a dense float32 device tensor [length][rot_dim/2][2]")
    _check("bfp8_rope_table", lib().bfp8_rope_table(
        out.data_ptr(), length, rot_dim, base, ROPE_SCALINGS[scaling], factor, original_length,
        _stream(out)))
    return out


def rope(x: torch.Tensor, table: torch.Tensor, positions: torch.Tensor = None,
         layout: str = "half", inverse: bool = False, out: torch.Tensor = None) -> torch.Tensor:
    """Turn the pairs of every head of x [tokens][heads][head_dim] (bfloat16 or
    float32) by their tokens' positions (int32 [tokens]; None: token t stands
    at t).  The rotated size is the table's.  ``inverse`` gives the gradient;
    ``out=x`` works in place.  See bfp8_rope."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    _check_heads(x, "x", tuple(DTYPES))
    if (table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32
            or not table.is_contiguous() or table.device != x.device):
        raise ValueError(f"table must be a dense float32 [length][rot_dim/2][2] on {x.device}")
    T, H, D = x.shape
    _check_i32(positions, "positions", T, x.device)
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    else:
        _check_heads(out, "out", (x.dtype,), x.device)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    xr, xh = _strides(x)
    yr, yh = _strides(out)
    _check("bfp8_rope", lib().bfp8_rope(
        x.data_ptr(), xr, xh, out.data_ptr(), yr, yh, DTYPES[x.dtype], T, H, D,
        2 * table.shape[1], ROPE_LAYOUTS[layout], table.data_ptr(), table.shape[0],
        _pointer(positions), int(inverse), _stream(x)))
    return out


# ---- attention --------------------------------------------------------------

_BF16 = (torch.bfloat16,)


def _shape(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale) -> AttentionShape:
    _check_heads(q, "q", _BF16)
    _check_heads(k, "k", _BF16, q.device)
    _check_heads(v, "v", _BF16, q.device)
    Tq, H, D = q.shape
    Tk, KV, Dk = k.shape
    if v.shape != k.shape:
        raise ValueError(f"k and v must have one shape, got {tuple(k.shape)} and {tuple(v.shape)}")
    if Dk != D:
        raise ValueError(f"q and k must have one head size, got {D} and {Dk}")
    if batch is None:
        given = [t.numel() - 1 for t in (cu_q, cu_k) if t is not None]
        given += [k_lens.numel()] if k_lens is not None else []
        batch = given[0] if given else 1
    _check_i32(cu_q, "cu_q", batch + 1, q.device)
    _check_i32(cu_k, "cu_k", batch + 1, q.device)
    _check_i32(k_lens, "k_lens", batch, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D) if D else 1.0
    return AttentionShape(batch, Tq, Tk, _pointer(cu_q), _pointer(cu_k), _pointer(k_lens), H, KV, D,
                          int(causal), scale)


def attention_workspace_bytes(q, k, v, cu_q=None, cu_k=None, k_lens=None, batch: int = None,
                              causal: bool = True, scale: float = None,
                              backward: bool = False) -> int:
    """Workspace bytes of attention_forward, or of attention_backward."""
    s = _shape(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    n = int(lib().bfp8_attention_workspace_bytes(ctypes.byref(s), int(backward)))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid attention shape")
    return n


def _workspace(shape, backward, given, device):
    n = int(lib().bfp8_attention_workspace_bytes(ctypes.byref(shape), int(backward)))
    if n == ctypes.c_size_t(-1).value:
        n = 0  # the call itself reports what is wrong with the shape
    if n and given is None:
        given = torch.empty((n,), dtype=torch.uint8, device=device)
    return given, (given.numel() * given.element_size() if given is not None else 0)


def _output(out, name, like, device):
    if out is None:
        return torch.empty(like.shape, dtype=torch.bfloat16, device=device)
    _check_heads(out, name, _BF16, device)
    if out.shape != like.shape:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)}")
    return out


def _check_lse(lse, heads, tokens, device):
    if (lse.shape != (heads, tokens) or lse.dtype != torch.float32 or not lse.is_contiguous()
            or lse.device != device):
        raise ValueError(f"lse must be a dense float32 [{heads}][{tokens}] on {device}")


def attention_forward(q, k, v, cu_q=None, cu_k=None, k_lens=None, batch: int = None,
                      causal: bool = True, scale: float = None, out: torch.Tensor = None,
                      lse: torch.Tensor = None, workspace: torch.Tensor = None):
    """Attention of q [Tq][H][D] over k, v [Tk][KV][D] (bfloat16, H a multiple
    of KV) -> (o [Tq][H][D], lse float32 [H][Tq]); see bfp8_attention_forward.

    cu_q, cu_k  int32 [batch+1]: first rows of the sequences; None: `batch`
                sequences (default 1) of equal length.
    k_lens      int32 [batch]: used rows of each sequence's keys; None: all.
    causal      query i of n sees keys 0 .. i + m - n of m.
    scale       default 1/sqrt(D).
    A workspace is allocated when the library asks for one and none is given."""
    s = _shape(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    out = _output(out, "out", q, q.device)
    if lse is None:
        lse = torch.empty((s.heads, s.total_q), dtype=torch.float32, device=q.device)
    else:
        _check_lse(lse, s.heads, s.total_q, q.device)
    workspace, nbytes = _workspace(s, False, workspace, q.device)
    _check("bfp8_attention_forward", lib().bfp8_attention_forward(
        ctypes.byref(s), _heads(q), _heads(k), _heads(v), _heads(out), lse.data_ptr(),
        _pointer(workspace), nbytes, _stream(q)))
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, k_lens=None,
                       batch: int = None, causal: bool = True, scale: float = None,
                       dq: torch.Tensor = None, dk: torch.Tensor = None, dv: torch.Tensor = None,
                       workspace: torch.Tensor = None):
    """Gradients (dq, dk, dv) of attention_forward for the gradient `dout` of
    its `out`, given the `lse` it returned and the same sequences, mask and
    scale; see bfp8_attention_backward."""
    s = _shape(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    for t, name in ((out, "out"), (dout, "dout")):
        _check_heads(t, name, _BF16, q.device)
        if t.shape != q.shape:
            raise ValueError(f"{name} must have the shape of q")
    _check_lse(lse, s.heads, s.total_q, q.device)
    dq = _output(dq, "dq", q, q.device)
    dk = _output(dk, "dk", k, q.device)
    dv = _output(dv, "dv", v, q.device)
    workspace, nbytes = _workspace(s, True, workspace, q.device)
    _check("bfp8_attention_backward", lib().bfp8_attention_backward(
        ctypes.byref(s), _heads(q), _heads(k), _heads(v), _heads(out), lse.data_ptr(),
        _heads(dout), _heads(dq), _heads(dk), _heads(dv), _pointer(workspace), nbytes,
        _stream(q)))
    return dq, dk, dv
