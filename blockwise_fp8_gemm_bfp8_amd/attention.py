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


# The calls below are short (a decode step's kernels take a few microseconds),
# so the marshalling is kept short, too: each tensor's sizes and strides are
# fetched once, and the current stream's handle without building a Stream.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: int):
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _heads(t: torch.Tensor, name: str, dtypes, device: int = None, shape=None):
    """Check a tensor of heads; returns its device, shape and bfp8_heads.
    The strides of axes with one entry do not matter and are given as head_dim,
    which every check passes whatever the other stride is."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and at != device:
        raise ValueError(f"{name} must be on device {device}, got {at}")
    size = t.shape
    if len(size) != 3:
        raise ValueError(f"{name} must be 3-D [tokens][heads][head_dim]")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(size)}")
    T, H, D = size
    row, head, one = t.stride()
    if one != 1 and D > 1 and T and H:
        raise ValueError(f"{name} must have unit stride along its last axis")
    if H <= 1:
        head = D
    if T <= 1:
        row = D
    return at, size, Heads(t.data_ptr(), row, head)


def _result(out, like: torch.Tensor, name: str, device: int, size):
    """The tensor of a result that has `like`'s shape (`size`) and dtype, a new
    dense one if `out` is None, and its bfp8_heads."""
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        _, H, D = size
        return out, Heads(out.data_ptr(), max(H, 1) * D, D)
    return out, _heads(out, name, (like.dtype,), device, size)[2]


def _check_i32(t, name: str, n: int, device: int):
    if t is None:
        return
    if (t.get_device() != device or t.dtype is not torch.int32 or t.dim() != 1
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a dense 1-D int32 tensor on device {device}")
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
    device, size, xh = _heads(x, "x", DTYPES)
    if (table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32
            or not table.is_contiguous() or table.get_device() != device):
        raise ValueError(f"table must be a dense float32 [length][rot_dim/2][2] on device {device}")
    T, H, D = size
    _check_i32(positions, "positions", T, device)
    out, yh = _result(out, x, "out", device, size)
    length, half, _ = table.shape
    _check("bfp8_rope", lib().bfp8_rope(
        xh.data, xh.row, xh.head, yh.data, yh.row, yh.head, DTYPES[x.dtype], T, H, D, 2 * half,
        ROPE_LAYOUTS[layout], table.data_ptr(), length, _pointer(positions), int(inverse),
        _stream_of(device)))
    return out


# ---- attention --------------------------------------------------------------

_BF16 = (torch.bfloat16,)
_INVALID = ctypes.c_size_t(-1).value  # bfp8_attention_workspace_bytes of an invalid shape


def _problem(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale):
    """Check the inputs; returns (device, bfp8_attention_shape, q, k, v as
    bfp8_heads, the shapes of q and of k)."""
    device, qs, qh = _heads(q, "q", _BF16)
    _, ks, kh = _heads(k, "k", _BF16, device)
    _, _, vh = _heads(v, "v", _BF16, device, ks)
    Tq, H, D = qs
    Tk, KV, Dk = ks
    if Dk != D:
        raise ValueError(f"q and k must have one head size, got {D} and {Dk}")
    if batch is None:
        batch = (cu_q.numel() - 1 if cu_q is not None else cu_k.numel() - 1 if cu_k is not None
                 else k_lens.numel() if k_lens is not None else 1)
    _check_i32(cu_q, "cu_q", batch + 1, device)
    _check_i32(cu_k, "cu_k", batch + 1, device)
    _check_i32(k_lens, "k_lens", batch, device)
    if scale is None:
        scale = 1.0 / math.sqrt(D) if D else 1.0
    s = AttentionShape(batch, Tq, Tk, _pointer(cu_q), _pointer(cu_k), _pointer(k_lens), H, KV,
                       D, int(causal), scale)
    if s.causal not in (0, 1):  # other bits are the library's BFP8_CLEAR_*
        raise ValueError(f"causal must be true or false, got {causal}")
    return device, s, qh, kh, vh, qs, ks


def attention_workspace_bytes(q, k, v, cu_q=None, cu_k=None, k_lens=None, batch: int = None,
                              causal: bool = True, scale: float = None,
                              backward: bool = False) -> int:
    """Workspace bytes of attention_forward, or of attention_backward."""
    _, s, *_ = _problem(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    n = lib().bfp8_attention_workspace_bytes(ctypes.byref(s), int(backward))
    if n == _INVALID:
        raise ValueError("invalid attention shape")
    return n


def _workspace(shape, backward, given, like):
    """(tensor or None, bytes)"""
    if given is None:
        n = lib().bfp8_attention_workspace_bytes(ctypes.byref(shape), backward)
        if n == 0 or n == _INVALID:  # the call itself reports what is wrong with a shape
            return None, 0
        given = torch.empty(n, dtype=torch.uint8, device=like.device)
        return given, n
    if given.get_device() != like.get_device() or not given.is_contiguous():
        raise ValueError(f"workspace must be a dense tensor on device {like.get_device()}")
    return given, given.numel() * given.element_size()


def _check_lse(lse, heads, tokens, device: int):
    if (lse.shape != (heads, tokens) or lse.dtype != torch.float32 or not lse.is_contiguous()
            or lse.get_device() != device):
        raise ValueError(f"lse must be a dense float32 [{heads}][{tokens}] on device {device}")


# BFP8_CLEAR_* in bfp8_attention_shape.causal
_CLEAR_O, _CLEAR_LSE, _CLEAR_DQ, _CLEAR_DK, _CLEAR_DV = (1 << i for i in range(8, 13))


def attention_forward(q, k, v, cu_q=None, cu_k=None, k_lens=None, batch: int = None,
                      causal: bool = True, scale: float = None, out: torch.Tensor = None,
                      lse: torch.Tensor = None, workspace: torch.Tensor = None,
                      zero_rest: bool = False):
    """Attention of q [Tq][H][D] over k, v [Tk][KV][D] (bfloat16, H a multiple
    of KV) -> (o [Tq][H][D], lse float32 [H][Tq]); see bfp8_attention_forward.

    cu_q, cu_k  int32 [batch+1]: first rows of the sequences; None: `batch`
                sequences (default 1) of equal length.
    k_lens      int32 [batch]: used rows of each sequence's keys; None: all.
    causal      query i of n sees keys 0 .. i + m - n of m.
    scale       default 1/sqrt(D).
    zero_rest   rows of no sequence (before cu_q[0], from cu_q[-1] on) become 0
                (lse: -inf) in a given out and lse, too; they always do in
                results that the call allocates.
    A workspace is allocated when the library asks for one and none is given."""
    device, s, qh, kh, vh, qs, _ = _problem(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    s.causal |= ((_CLEAR_O if out is None or zero_rest else 0)
                 | (_CLEAR_LSE if lse is None or zero_rest else 0))
    out, oh = _result(out, q, "out", device, qs)
    if lse is None:
        lse = torch.empty(qs[1], qs[0], dtype=torch.float32, device=q.device)
    else:
        _check_lse(lse, s.heads, s.total_q, device)
    workspace, nbytes = _workspace(s, 0, workspace, q)
    _check("bfp8_attention_forward", lib().bfp8_attention_forward(
        ctypes.byref(s), qh, kh, vh, oh, lse.data_ptr(), _pointer(workspace), nbytes,
        _stream_of(device)))
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, k_lens=None,
                       batch: int = None, causal: bool = True, scale: float = None,
                       dq: torch.Tensor = None, dk: torch.Tensor = None, dv: torch.Tensor = None,
                       workspace: torch.Tensor = None, zero_rest: bool = False):
    """Gradients (dq, dk, dv) of attention_forward for the gradient `dout` of
    its `out`, given the `lse` it returned and the same sequences, mask and
    scale; see bfp8_attention_backward.  Rows of no sequence are zero in
    gradients that the call allocates and, with `zero_rest`, in given ones."""
    device, s, qh, kh, vh, qs, ks = _problem(q, k, v, cu_q, cu_k, k_lens, batch, causal, scale)
    _, _, oh = _heads(out, "out", _BF16, device, qs)
    _, _, doh = _heads(dout, "dout", _BF16, device, qs)
    _check_lse(lse, s.heads, s.total_q, device)
    s.causal |= ((_CLEAR_DQ if dq is None or zero_rest else 0)
                 | (_CLEAR_DK if dk is None or zero_rest else 0)
                 | (_CLEAR_DV if dv is None or zero_rest else 0))
    dq, dqh = _result(dq, q, "dq", device, qs)
    dk, dkh = _result(dk, k, "dk", device, ks)
    dv, dvh = _result(dv, v, "dv", device, ks)
    workspace, nbytes = _workspace(s, 1, workspace, q)
    _check("bfp8_attention_backward", lib().bfp8_attention_backward(
        ctypes.byref(s), qh, kh, vh, oh, lse.data_ptr(), doh, dqh, dkh, dvh, _pointer(workspace),
        nbytes, _stream_of(device)))
    return dq, dk, dv
