"""The binding of include/zero_linear.h: the layer products on the flat
16-bit buffers and the counter-based dropout.

    w = weights[off:off + n * k].view(n, k)       # the all-gather buffer
    zero_linear(x, w, y, bias=b, act=ZERO_ACT_GELU_TANH, z=z)
    zero_linear_dgrad(dy2, w2, dz, act=ZERO_ACT_GELU_TANH, z=z)
    zero_linear_wgrad(dz, x, row[off:off + n * k].view(n, k), db=...)

Matrices are 2-D tensors or views whose rows are contiguous; any row stride
and any element alignment is taken.  Dimensions come from the tensors and are
checked against each other before anything is launched.
"""
import ctypes
from dataclasses import dataclass
from typing import Any

import torch

from . import _buf, _check, _lib, _torch_stream, ZERO_BF16, ZERO_FP16, ZERO_FP32

ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU, ZERO_ACT_GELU_TANH, ZERO_ACT_SILU = range(5)
ZERO_LINEAR, ZERO_LINEAR_DGRAD, ZERO_LINEAR_WGRAD = range(3)

_CODE = {torch.bfloat16: ZERO_BF16, torch.float16: ZERO_FP16, torch.float32: ZERO_FP32}
_WIDTH = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4}


class _DropoutParams(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("row0", ctypes.c_int64), ("step", ctypes.c_void_p)]


@dataclass
class ZeroDropout:
    """Dropout D: the mask is a function of seed, offset (+ *step, an int64
    GPU tensor such as new_step_counter()'s, read when the kernel runs), row
    (counted from row0) and column; see zero_linear.h for the exact bits."""
    p: float
    seed: int = 0
    offset: int = 0
    row0: int = 0
    step: Any = None

    def _c(self, device):
        return _DropoutParams(self.p, self.seed & 0xFFFFFFFFFFFFFFFF,
                              self.offset & 0xFFFFFFFFFFFFFFFF, self.row0,
                              _buf(self.step, "drop.step", 1, torch.int64, device))


def _declare(L):
    vp, i64, i32, enum = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    dp = ctypes.POINTER(_DropoutParams)
    L.zero_linear_workspace_bytes.argtypes = [enum, i64, i64, i64]
    L.zero_linear_workspace_bytes.restype = i64
    L.zero_linear.argtypes = [vp, enum, i64, vp, i64, vp, i64, i64, i64, enum, dp, vp, i64, vp,
                              enum, i64, vp, i64, vp, i64, vp]
    L.zero_linear.restype = enum
    L.zero_linear_dgrad.argtypes = [vp, enum, i64, vp, i64, i64, i64, i64, enum, vp, i64, dp, vp,
                                    i64, vp, enum, i64, vp, i64, vp]
    L.zero_linear_dgrad.restype = enum
    L.zero_linear_wgrad.argtypes = [vp, enum, i64, vp, i64, i64, i64, i64, vp, enum, i64, vp, i32,
                                    vp, i64, vp]
    L.zero_linear_wgrad.restype = enum
    L.zero_dropout.argtypes = [vp, enum, i64, i64, i64, dp, vp, i64, vp, i64, vp]
    L.zero_dropout.restype = enum


_declare(_lib)


def _mat(t, what: str, rows=None, cols=None, dtype=None, device=None):
    """(address, row stride) of a GPU matrix with contiguous rows, its shape,
    type and device as given (None: whatever they are)."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: a GPU tensor is required")
    if t.dim() != 2:
        raise TypeError(f"{what}: a 2-D tensor is required, got {t.dim()}-D")
    if dtype is None:
        if t.dtype not in _CODE:
            raise TypeError(f"{what}: bfloat16, float16 or float32 expected, got {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, the call's tensors are on {device}")
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{what}: [{rows if rows is not None else 'any'}]"
                         f"[{cols if cols is not None else 'any'}] expected, got [{r}][{c}]")
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        raise TypeError(f"{what}: rows of contiguous elements are required")
    if r > 1 and s0 < c:
        raise TypeError(f"{what}: rows that do not overlap are required (row stride {s0})")
    return t.data_ptr(), (s0 if r > 1 else max(c, 1))


def _optional(t, what, rows, cols, dtype, device):
    return (None, cols) if t is None else _mat(t, what, rows, cols, dtype, device)


def _out_type(t, dt, what):
    if t.dtype != dt and t.dtype != torch.float32:
        raise TypeError(f"{what}: {dt} or torch.float32 expected, got {t.dtype}")
    return t.dtype


def _in_type(t, what):
    dt = getattr(t, "dtype", None)
    if dt != torch.bfloat16 and dt != torch.float16:
        raise TypeError(f"{what}: 16-bit (bfloat16 or float16) tensor expected, got {dt}")
    return dt


def zero_linear_workspace_bytes(op: int, m: int, n: int, k: int) -> int:
    """Bytes of device workspace a product needs: op ZERO_LINEAR,
    ZERO_LINEAR_DGRAD or ZERO_LINEAR_WGRAD with W [n][k] and m rows."""
    b = _lib.zero_linear_workspace_bytes(op, m, n, k)
    if b < 0:
        raise ValueError(f"zero_linear_workspace_bytes: op {op}, m {m}, n {n}, k {k} out of range")
    return b


def _scratch(op, m, n, k, workspace, stream, device):
    """(address, bytes) of the product's workspace: the caller's, or a new
    one allocated on the call's stream (so that freeing it on return is
    ordered after the kernels)."""
    need = _lib.zero_linear_workspace_bytes(op, m, n, k)
    if need <= 0:
        return None, 0
    if workspace is None:
        with torch.cuda.stream(_torch_stream(stream, device)):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace: {need} bytes needed, the tensor holds {have}")
    return _buf(workspace, "workspace", 0, device=device), have


def _call(fn, what, device, stream, *args):
    s = _torch_stream(stream, device).cuda_stream
    if device.index is not None and device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _check(fn(*args, s), what)
    else:
        _check(fn(*args, s), what)


def zero_linear(x, w, y, bias=None, act: int = ZERO_ACT_NONE, drop=None, residual=None, z=None,
                stream=None, workspace=None):
    """y = residual + D(act(z)), z = x w^T + bias: x [m][k] and w [n][k] bf16
    or fp16, y [m][n] of that type or fp32, residual of y's type (it may be y
    itself), z (optional) [m][n] of x's type.  drop: a ZeroDropout or None.
    A workspace tensor is allocated where one is needed unless one of
    zero_linear_workspace_bytes(ZERO_LINEAR, m, n, k) bytes is passed."""
    dt, d = _in_type(x, "x"), x.device
    px, ldx = _mat(x, "x", dtype=dt)
    m, k = x.shape
    pw, ldw = _mat(w, "w", None, k, dt, d)
    n = w.shape[0]
    py, ldy = _mat(y, "y", m, n, _out_type(y, dt, "y"), d)
    pr, ldr = _optional(residual, "residual", m, n, y.dtype, d)
    pz, ldz = _optional(z, "z", m, n, dt, d)
    ws, nb = _scratch(ZERO_LINEAR, m, n, k, workspace, stream, d)
    _call(_lib.zero_linear, "zero_linear", d, stream, px, _CODE[dt], ldx, pw, ldw,
          _buf(bias, "bias", n, dt, d), m, n, k, act,
          None if drop is None else ctypes.byref(drop._c(d)), pr, ldr, py, _CODE[y.dtype], ldy,
          pz, ldz, ws, nb)


def zero_linear_dgrad(dy, w, dx, act: int = ZERO_ACT_NONE, z=None, drop=None, residual=None,
                      stream=None, workspace=None):
    """dx = residual + D(act'(z) * (dy w)): dy [m][n] and w [n][k] bf16 or
    fp16, dx [m][k] of that type or fp32, residual of dx's type (it may be dx
    itself).  act, z [m][k] and drop are those of the call that made this
    layer's input.  Workspace as for zero_linear."""
    dt, d = _in_type(dy, "dy"), dy.device
    py, lddy = _mat(dy, "dy", dtype=dt)
    m, n = dy.shape
    pw, ldw = _mat(w, "w", n, None, dt, d)
    k = w.shape[1]
    px, lddx = _mat(dx, "dx", m, k, _out_type(dx, dt, "dx"), d)
    pr, ldr = _optional(residual, "residual", m, k, dx.dtype, d)
    pz, ldz = _optional(z, "z", m, k, dt, d)
    ws, nb = _scratch(ZERO_LINEAR_DGRAD, m, n, k, workspace, stream, d)
    _call(_lib.zero_linear_dgrad, "zero_linear_dgrad", d, stream, py, _CODE[dt], lddy, pw, ldw, m,
          n, k, act, pz, ldz, None if drop is None else ctypes.byref(drop._c(d)), pr, ldr, px,
          _CODE[dx.dtype], lddx, ws, nb)


def zero_linear_wgrad(dy, x, dw, db=None, accumulate: bool = False, stream=None, workspace=None):
    """dw (+)= dy^T x and db (+)= the column sums of dy: dy [m][n] and x
    [m][k] bf16 or fp16, dw [n][k] and db (n elements) of that type or fp32,
    usually places in a flat gradient row; accumulate adds to what they hold
    (a later micro-batch).  Workspace as for zero_linear."""
    dt, d = _in_type(dy, "dy"), dy.device
    py, lddy = _mat(dy, "dy", dtype=dt)
    m, n = dy.shape
    px, ldx = _mat(x, "x", m, None, dt, d)
    k = x.shape[1]
    pg, lddw = _mat(dw, "dw", n, k, _out_type(dw, dt, "dw"), d)
    ws, nb = _scratch(ZERO_LINEAR_WGRAD, m, n, k, workspace, stream, d)
    _call(_lib.zero_linear_wgrad, "zero_linear_wgrad", d, stream, py, _CODE[dt], lddy, px, ldx, m,
          n, k, pg, _CODE[dw.dtype], lddw, _buf(db, "db", n, dw.dtype, d), int(bool(accumulate)),
          ws, nb)


def zero_dropout(x, y, drop, residual=None, stream=None):
    """y = residual + D(x) (2-D, bf16, fp16 or fp32; y may be x or residual
    itself).  The backward pass is the same call on the gradient."""
    px, ldx = _mat(x, "x")
    d, (m, n) = x.device, x.shape
    py, ldy = _mat(y, "y", m, n, x.dtype, d)
    pr, ldr = _optional(residual, "residual", m, n, x.dtype, d)
    if drop is None:
        raise TypeError("drop: a ZeroDropout is required")
    _call(_lib.zero_dropout, "zero_dropout", d, stream, px, _CODE[x.dtype], ldx, m, n,
          ctypes.byref(drop._c(d)), pr, ldr, py, ldy)
