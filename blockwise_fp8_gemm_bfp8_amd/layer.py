"""Binding of include/bfp8_layer.h: the RMS norm with the residual's addition,
the gated activation, both with E4M3 codes of their results, their gradients,
and the norm and clipping of many gradients.

Argument marshalling only, as in the package's other calls: every step runs in
the HIP kernels of libbfp8.so on the current stream of the tensors' device.
"""

import ctypes

import torch

from . import DTYPES, BFP8Error, GradJob, _padded_empty, _scale_bytes, lib
from .attention import _pointer, _stream_of

_ANY = tuple(DTYPES)
CODE_FORMATS = {"fp32": 0, "mx128": 1, "mx32": 2}  # hotpath's scale formats
_INVALID = ctypes.c_size_t(-1).value


# A generation step's kernels take a few microseconds, so the marshalling is kept
# short: results without padding are allocated without a view, and the device is
# changed only where the current one is another.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, device, *args):
    """The library's call `name` on the current stream of `device`."""
    fn = getattr(lib(), name)
    if _current_device() == device:
        code = fn(*args, _stream_of(device))
    else:  # launches go to the current device
        with torch.cuda.device(device):
            code = fn(*args, _stream_of(device))
    if code:
        raise BFP8Error(name, code)


def _matrix(t, name, device=None, shape=None, dtype=None):
    """Check a matrix of activations; returns its row stride (of no account, and
    given as one that passes, where there is one row at most)."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and at != device:
        raise ValueError(f"{name} must be on device {device}, got {at}")
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{name} must be 2-D")
    if dtype is None:
        if t.dtype not in DTYPES:
            raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    elif t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(size)}")
    row, one = t.stride()
    if one != 1 and size[1] > 1:
        raise ValueError(f"{name} must have unit stride along its last axis")
    return row if size[0] > 1 else max(-(-size[1] // 16) * 16, 16)


def _rows_empty(rows, cols, dtype, device, align):
    """_padded_empty, without its view where there is nothing to pad."""
    if cols % align == 0 and cols:
        return torch.empty(rows, cols, dtype=dtype, device=device)  # sooner parsed than a tuple
    return _padded_empty(rows, cols, dtype, device, align)


def _result(out, like, name, device):
    """The matrix of a result that has `like`'s shape and dtype, a new one if
    `out` is None, and its row stride."""
    if out is None:
        rows, cols = like.shape
        out = _rows_empty(rows, cols, like.dtype, like.device, 16 // like.element_size())
        return out, out.stride(0)
    return out, _matrix(out, name, device, like.shape, like.dtype)


def _vector(t, name, n, device, dtypes=(torch.float32,)):
    if t.shape != (n,) or t.dtype not in dtypes or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a dense {' or '.join(str(d) for d in dtypes)} [{n}] on "
                         f"device {device}")


def _codes(t, name, rows, cols, device, place):
    """The matrix of codes, a new one if `t` is None, and its row stride."""
    if t is None:
        t = _rows_empty(rows, cols, torch.uint8, place, 16)
        return t, t.stride(0)
    return t, _matrix(t, name, device, (rows, cols), torch.uint8)


def _scales(t, name, rows, cols, scales, device, place):
    """The scales of rows x cols codes in the layout of the format."""
    shape = (rows, cols // 32) if scales == "mx32" else (cols // 128, rows)
    if t is None:
        if scales == "fp32":
            return torch.empty(*shape, dtype=torch.float32, device=place)
        return _scale_bytes(*shape, place)
    dtype = torch.float32 if scales == "fp32" else torch.uint8
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a dense {dtype} [{shape[0]}][{shape[1]}] on device {device}")
    return t


def _codes_out(rows, cols, scales, transposed, given, like, device):
    """([q, s] or [q, s, qt, st], their arguments) of a rows x cols result;
    `given`: q, s, qt, st or Nones."""
    fmt = CODE_FORMATS.get(scales)
    if fmt is None:
        raise ValueError(f"scales must be one of {sorted(CODE_FORMATS)}")
    q, s, qt, st = given
    if not transposed and (qt is not None or st is not None):
        raise ValueError("qt and st are written with transposed=True only")
    place = like.device
    q, ldq = _codes(q, "q", rows, cols, device, place)
    s = _scales(s, "s", rows, cols, scales, device, place)
    if not transposed:
        return [q, s], (fmt, q.data_ptr(), ldq, s.data_ptr(), None, 0, None)
    qt, ldqt = _codes(qt, "qt", cols, rows, device, place)
    st = _scales(st, "st", cols, rows, scales, device, place)
    return [q, s, qt, st], (fmt, q.data_ptr(), ldq, s.data_ptr(), qt.data_ptr(), ldqt,
                            st.data_ptr())


# ---- RMS norm -----------------------------------------------------------------

def _norm_inputs(x, weight, residual, sum_out, rstd):
    device = x.get_device()
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    _vector(weight, "weight", cols, device, _ANY)
    ldr = lds = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", device, x.shape, x.dtype)
        sum_out, lds = _result(sum_out, x, "sum_out", device)
    elif sum_out is not None:
        raise ValueError("sum_out is the sum with a residual: there is none")
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    else:
        _vector(rstd, "rstd", rows, device)
    head = (x.data_ptr(), ldx, _pointer(residual), ldr, weight.data_ptr(), DTYPES[weight.dtype],
            DTYPES[x.dtype], rows, cols)
    return device, head, sum_out, lds, rstd


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor = None,
            eps: float = 1e-6, out: torch.Tensor = None, sum_out: torch.Tensor = None,
            rstd: torch.Tensor = None):
    """r = x + residual (x without one), y = r / sqrt(mean(r^2) + eps) * weight for
    rows x [rows][cols] (bfloat16 or float32) -> (y, r, rstd float32 [rows]).
    r and rstd are what the gradient needs; ``sum_out=residual`` adds in place (and
    ``out=x`` without a residual gives r up).  See bfp8_rmsnorm."""
    device, head, sum_out, lds, rstd = _norm_inputs(x, weight, residual, sum_out, rstd)
    out, ldy = _result(out, x, "out", device)
    _call("bfp8_rmsnorm", device, *head, eps, _pointer(sum_out), lds, out.data_ptr(), ldy,
          rstd.data_ptr())
    return out, x if residual is None else sum_out, rstd


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor = None,
                     eps: float = 1e-6, scales: str = "fp32", transposed: bool = False,
                     q=None, s=None, qt=None, st=None, sum_out: torch.Tensor = None,
                     rstd: torch.Tensor = None):
    """rmsnorm with E4M3 codes of y in place of y -> (q, s, r, rstd), or with
    ``transposed`` (q, s, qt, st, r, rstd): both layouts, for a linear's forward
    and weight gradient.  ``scales`` is hotpath's format: "fp32" (as
    quantize_act_dual_kmajor writes them), "mx128" (quantize_mx_act_dual_kmajor)
    or "mx32" (quantize_mx_act_dual, group 32).  See bfp8_rmsnorm_quantize."""
    device, head, sum_out, lds, rstd = _norm_inputs(x, weight, residual, sum_out, rstd)
    out, args = _codes_out(*x.shape, scales, transposed, (q, s, qt, st), x, device)
    _call("bfp8_rmsnorm_quantize", device, *head, eps, _pointer(sum_out), lds, rstd.data_ptr(),
          *args)
    return (*out, x if residual is None else sum_out, rstd)


def rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    n = lib().bfp8_rmsnorm_backward_workspace_bytes(rows, cols)
    if n == _INVALID:
        raise ValueError("invalid sizes")
    return n


def rmsnorm_backward(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dsum: torch.Tensor = None, dx: torch.Tensor = None,
                     dweight: torch.Tensor = None, workspace: torch.Tensor = None):
    """(dx, dweight float32 [cols]) for the gradient dy of rmsnorm's y, its r and
    rstd, and the gradient ``dsum`` that arrives at r itself; dx is the gradient
    of x and of the residual.  See bfp8_rmsnorm_backward."""
    device = dy.get_device()
    lddy = _matrix(dy, "dy")
    rows, cols = dy.shape
    ldr = _matrix(r, "r", device, dy.shape, dy.dtype)
    _vector(weight, "weight", cols, device, _ANY)
    _vector(rstd, "rstd", rows, device)
    lds = _matrix(dsum, "dsum", device, dy.shape, dy.dtype) if dsum is not None else 0
    dx, lddx = _result(dx, dy, "dx", device)
    if dweight is None:
        dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
    else:
        _vector(dweight, "dweight", cols, device)
    if workspace is None:
        nbytes = lib().bfp8_rmsnorm_backward_workspace_bytes(rows, cols)
        if nbytes != _INVALID:  # the call itself reports what is wrong with the sizes
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    nbytes = _workspace_size(workspace, device)
    _call("bfp8_rmsnorm_backward", device, dy.data_ptr(), lddy, r.data_ptr(), ldr, weight.data_ptr(),
          DTYPES[weight.dtype], rstd.data_ptr(), _pointer(dsum), lds, DTYPES[dy.dtype], rows, cols,
          dx.data_ptr(), lddx, dweight.data_ptr(), _pointer(workspace), nbytes)
    return dx, dweight


def _workspace_size(t, device):
    if t is None:
        return 0
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a dense tensor on device {device}")
    return t.numel() * t.element_size()


# ---- gated activation -----------------------------------------------------------

def _glu_inputs(gate, up, dh=None):
    device = gate.get_device()
    ldg = _matrix(gate, "gate")
    ldu = _matrix(up, "up", device, gate.shape, gate.dtype)
    head = (gate.data_ptr(), ldg, up.data_ptr(), ldu, DTYPES[gate.dtype], *gate.shape)
    if dh is not None:
        head = (dh.data_ptr(), _matrix(dh, "dh", device, gate.shape, gate.dtype), *head)
    return device, head


def swiglu(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor = None) -> torch.Tensor:
    """silu(gate) * up for gate, up [rows][cols] (bfloat16 or float32), usually the
    halves of one projection's rows.  See bfp8_swiglu."""
    device, head = _glu_inputs(gate, up)
    out, ldh = _result(out, gate, "out", device)
    _call("bfp8_swiglu", device, *head, out.data_ptr(), ldh)
    return out


def swiglu_quantize(gate: torch.Tensor, up: torch.Tensor, scales: str = "fp32",
                    transposed: bool = False, q=None, s=None, qt=None, st=None):
    """swiglu with E4M3 codes of its result in place of it -> (q, s), or with
    ``transposed`` (q, s, qt, st); ``scales`` as for rmsnorm_quantize.  See
    bfp8_swiglu_quantize."""
    device, head = _glu_inputs(gate, up)
    out, args = _codes_out(*gate.shape, scales, transposed, (q, s, qt, st), gate, device)
    _call("bfp8_swiglu_quantize", device, *head, *args)
    return tuple(out)


def swiglu_backward(dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                    dgate: torch.Tensor = None, dup: torch.Tensor = None):
    """(dgate, dup) for the gradient dh of swiglu(gate, up).  See bfp8_swiglu_backward."""
    device, head = _glu_inputs(gate, up, dh)
    dgate, ldg = _result(dgate, gate, "dgate", device)
    dup, ldu = _result(dup, gate, "dup", device)
    _call("bfp8_swiglu_backward", device, *head, dgate.data_ptr(), ldg, dup.data_ptr(), ldu)
    return dgate, dup


def swiglu_backward_quantize(dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                             scales: str = "fp32", transposed: bool = False, q=None, s=None,
                             qt=None, st=None):
    """E4M3 codes of the rows [dgate | dup] (2 cols wide), the gradient of a
    projection whose rows are [gate | up] -> (q, s), or with ``transposed``
    (q, s, qt, st).  See bfp8_swiglu_backward_quantize."""
    device, head = _glu_inputs(gate, up, dh)
    rows, cols = gate.shape
    out, args = _codes_out(rows, 2 * cols, scales, transposed, (q, s, qt, st), gate, device)
    _call("bfp8_swiglu_backward_quantize", device, *head, *args)
    return tuple(out)


# ---- the norm of all gradients, and clipping ----------------------------------------

def _span(at, rows, cols, ld, size, *_):
    """(first byte, rows, bytes a row, bytes from row to row) of a matrix."""
    if rows == 1 or ld == cols:
        rows, cols, ld = 1, rows * cols, rows * cols
    return at, rows, cols * size, ld * size


def _meet(a, b):
    """Whether two such places share a byte."""
    if a[1] > b[1]:
        a, b = b, a
    (start, rows, width, ld), (other, other_rows, other_width, other_ld) = a, b

    def row_meets(at, low, high):
        # rows m of `low` to `high`, at m ld, of the other place: one around byte `at`?
        first = (at - other_width - other) // other_ld + 1
        last = -((other - at - width) // other_ld) - 1
        return max(first, low) <= min(last, high)

    if ld == other_ld:  # only the difference of two rows' numbers counts
        return row_meets(start, 1 - rows, other_rows - 1)
    return any(row_meets(start + i * ld, 0, other_rows - 1) for i in range(rows))


def _refuse_overlaps(places):
    """What a job writes is its own: neither another's nor a shifted part of its own
    gradient.  places: (first byte, rows, cols, row stride, bytes a value, number, "grads"
    or "out")."""
    reach, end = [], 0  # the places since the last gap, and where they end
    for place in sorted(places):
        at, rows, cols, ld, size, i, kind = place
        if at >= end:
            reach.clear()
        for p in reach:
            if (kind == "out" or p[6] == "out") and _meet(_span(*p), _span(*place)):
                raise ValueError(f"{p[6]}[{p[5]}] and {kind}[{i}] share memory: one writes what the other "
                                 "holds")
        reach.append(place)
        end = max(end, at + ((rows - 1) * ld + cols) * size)


class GradClip:
    """The global norm and the clipping of a fixed list of gradients (bfloat16 or
    float32, dense, or 2-D with rows of unit stride) whose buffers stay: the
    table of their places is made once.

    out   where the clipped gradients go, tensors of the same shapes and types;
          None: in place.  Memory that is written twice, or that is another
          gradient's or a shifted part of the same one, is refused: a gradient
          is listed once.  (grad_norm writes nothing and counts it twice.)

    norm() is the square root of the sum of all squares (float32 0-d device
    tensor); clip(max_norm) scales by max_norm / norm where the norm exceeds
    max_norm.  Neither synchronises.  A norm over several ranks: sum norm()**2
    over them and give its root to clip()."""

    def __init__(self, grads, out=None, _clips=True):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients but {len(self.out)} outputs")
        if not self.grads:
            raise ValueError("no gradients")
        self.device, self._device = self.grads[0].get_device(), self.grads[0].device
        self._jobs, places = (GradJob * len(self.grads))(), []
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            rows, cols, ldg = self._place(g, f"grads[{i}]")
            if o is not g and (o.shape != g.shape or o.dtype != g.dtype):
                raise ValueError(f"out[{i}] must be {g.dtype} {list(g.shape)}, got {o.dtype} "
                                 f"{list(o.shape)}")
            at, size, dtype = g.data_ptr(), g.element_size(), DTYPES[g.dtype]
            if o is g:
                out, ldo = at, ldg
            else:
                out = o.data_ptr()
                orows, ocols, ldo = self._place(o, f"out[{i}]")
                if (orows, ocols) != (rows, cols):  # one of the two is dense, the other strided
                    rows, cols = g.shape
                    ldg, ldo = (t.stride(0) if rows > 1 else cols for t in (g, o))
            self._jobs[i] = GradJob(at, out, rows, cols, ldg, ldo, dtype)
            if rows and cols:
                places.append((out, rows, cols, ldo, size, i, "out"))
                if out != at or ldo != ldg:
                    places.append((at, rows, cols, ldg, size, i, "grads"))
        if _clips:
            _refuse_overlaps(places)
        n = lib().bfp8_grad_norm_workspace_bytes(self._jobs, len(self._jobs))
        if n == _INVALID:
            raise ValueError("invalid gradients")
        self._bytes = n

    def _place(self, t, name):
        """(rows, cols, row stride)"""
        if t.get_device() != self.device or self.device < 0:
            raise ValueError(f"{name} must be a device tensor, and all on one device")
        if t.dtype not in DTYPES:
            raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
        if t.is_contiguous():
            return 1, t.numel(), t.numel()
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
            return t.shape[0], t.shape[1], t.stride(0)
        raise ValueError(f"{name} must be dense, or 2-D with rows of unit stride")

    @property
    def workspace_bytes(self) -> int:
        return self._bytes

    def _norm_out(self, out, workspace):
        """The norm's tensor, the workspace's pointer and its bytes; either is
        allocated when none is given."""
        if out is None:
            out = torch.empty((), dtype=torch.float32, device=self._device)
        else:
            self._check_norm(out, "out")
        if workspace is None:
            workspace = torch.empty(self._bytes, dtype=torch.uint8, device=self._device)
            return out, workspace, self._bytes
        return out, workspace, _workspace_size(workspace, self.device)

    def norm(self, out: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
        """The norm of the gradients as they are now."""
        out, workspace, nbytes = self._norm_out(out, workspace)
        _call("bfp8_grad_norm", self.device, self._jobs, len(self._jobs), out.data_ptr(),
              workspace.data_ptr(), nbytes)
        return out

    def _check_norm(self, t, name):
        if t.dtype != torch.float32 or t.numel() != 1 or t.get_device() != self.device:
            raise ValueError(f"{name} must be one float32 on device {self.device}")

    def clip(self, max_norm: float, norm: torch.Tensor = None,
             workspace: torch.Tensor = None) -> torch.Tensor:
        """Writes the clipped gradients to `out`; returns the norm they were
        clipped by: `norm`, or this call's own."""
        if norm is not None:
            self._check_norm(norm, "norm")
            _call("bfp8_grad_clip", self.device, self._jobs, len(self._jobs), norm.data_ptr(),
                  max_norm)
            return norm
        norm, workspace, nbytes = self._norm_out(None, workspace)
        _call("bfp8_grad_norm_clip", self.device, self._jobs, len(self._jobs), norm.data_ptr(),
              max_norm, workspace.data_ptr(), nbytes)
        return norm


def grad_norm(grads) -> torch.Tensor:
    """The global norm of the gradients; see GradClip."""
    return GradClip(grads, _clips=False).norm()


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Clips the gradients (in place, or into `out`) to max_norm taken together;
    returns their norm before.  For gradients whose buffers stay, keep a GradClip."""
    return GradClip(grads, out).clip(max_norm)
