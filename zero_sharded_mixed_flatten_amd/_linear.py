"""The binding of include/zero_linear.h: the layer products on the flat
16-bit buffers and the counter-based dropout.

    w = weights[off:off + n * k].view(n, k)       # the all-gather buffer
    zero_linear(x, w, y, bias=b, act=ZERO_ACT_GELU_TANH, z=z)
    zero_linear_dgrad(dy2, w2, dz, act=ZERO_ACT_GELU_TANH, z=z)
    zero_linear_wgrad(dz, x, row[off:off + n * k].view(n, k), db=...)

Matrices are 2-D tensors or views whose rows are contiguous; any row stride
and any element alignment is taken.  Dimensions come from the tensors and are
checked against each other before anything is launched.

As everywhere in the binding the calls read and write through plain addresses:
autograd records none of them, whatever requires_grad says, and a tensor's
version counter does not move when a call writes into it, so autograd does not
notice if it had saved that tensor.  The backward pass is the caller's own
zero_linear_dgrad, zero_linear_wgrad and zero_dropout.
"""
import ctypes
from dataclasses import dataclass
from typing import Any

import torch

from . import _buf, _check, _lib, _torch_stream, ZERO_BF16, ZERO_FP16, ZERO_FP32

ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU, ZERO_ACT_GELU_TANH, ZERO_ACT_SILU = range(5)
ZERO_LINEAR, ZERO_LINEAR_DGRAD, ZERO_LINEAR_WGRAD = range(3)

_CODE = {torch.bfloat16: ZERO_BF16, torch.float16: ZERO_FP16, torch.float32: ZERO_FP32}


class _DropoutParams(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("row0", ctypes.c_int64), ("step", ctypes.c_void_p)]


@dataclass
class ZeroDropout:
    """Dropout D: the mask is a function of seed, offset (+ *step, an int64
    GPU tensor such as new_step_counter()'s, read when the kernel runs), row
    (counted from row0) and column; see zero_linear.h for the exact bits.
    Calls of one seed whose offset + *step are equal draw the same mask, those
    left at the defaults too: layers that should not share one take seeds of
    their own, or offsets that the counter never bridges (layer << 32 serves
    2^32 steps)."""
    p: float
    seed: int = 0
    offset: int = 0
    row0: int = 0
    step: Any = None

    def _c(self, device):
        return _DropoutParams(self.p, self.seed & 0xFFFFFFFFFFFFFFFF,
                              self.offset & 0xFFFFFFFFFFFFFFFF, self.row0,
                              None if self.step is None else
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


def _mat(t, what, shape, dtype, dev):
    """(address, row stride) of a GPU matrix of this shape and type on device
    number dev, with contiguous rows."""
    if t.is_cuda and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        s0, s1 = t.stride()
        if s1 == 1 and s0 >= shape[1]:
            return t.data_ptr(), s0
    return _odd_mat(t, what, shape, dtype, dev)


def _odd_mat(t, what, shape, dtype, dev):
    """_mat for single rows and columns, whose strides mean nothing; else the refusal."""
    if not t.is_cuda:
        raise TypeError(f"{what}: a GPU tensor is required")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, the call's tensors are on cuda:{dev}")
    if t.dim() != 2:
        raise TypeError(f"{what}: a 2-D tensor is required, got {t.dim()}-D")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: {tuple(shape)} expected, got {tuple(t.shape)}")
    (r, c), (s0, s1) = t.shape, t.stride()
    if c > 1 and s1 != 1:
        raise TypeError(f"{what}: rows of contiguous elements are required")
    if r > 1 and s0 < c:
        raise TypeError(f"{what}: rows that do not overlap are required (row stride {s0})")
    return t.data_ptr(), (s0 if r > 1 else max(c, 1))


def _shape(t, what):
    """a matrix argument's own shape and device number"""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: a GPU tensor is required")
    if t.dim() != 2:
        raise TypeError(f"{what}: a 2-D tensor is required, got {t.dim()}-D")
    return t.shape


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
    """(tensor, address, bytes) of the product's workspace: the caller's, or a
    new one allocated on the call's stream.  The caller holds the tensor until
    its kernels are enqueued: freed after that, its block is reused in the
    stream's order, behind them; freed before, another thread could be handed
    it first (the library is called without the interpreter's lock)."""
    if workspace is None:
        need = _lib.zero_linear_workspace_bytes(op, m, n, k)
        if need <= 0:
            return None, None, 0
        with torch.cuda.stream(_torch_stream(stream, device)):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    return workspace, _buf(workspace, "workspace", 0, device=device).value, \
        workspace.numel() * workspace.element_size()


def _call(fn, what, dev, stream, *args):
    """fn(*args, stream) with the tensors' device current; None is that
    device's current stream."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status, what)


def zero_linear(x, w, y, bias=None, act: int = ZERO_ACT_NONE, drop=None, residual=None, z=None,
                stream=None, workspace=None):
    """y = residual + D(act(z)), z = x w^T + bias: x [m][k] and w [n][k] bf16
    or fp16, y [m][n] of that type or fp32, residual of y's type (it may be y
    itself), z (optional) [m][n] of x's type.  drop: a ZeroDropout or None.
    A workspace tensor is allocated where one is needed unless one of
    zero_linear_workspace_bytes(ZERO_LINEAR, m, n, k) bytes is passed."""
    dt = _in_type(x, "x")
    m, k = _shape(x, "x")
    n = _shape(w, "w")[0]
    dev, out, yt = x.get_device(), (m, n), _out_type(y, dt, "y")
    px, ldx = _mat(x, "x", (m, k), dt, dev)
    pw, ldw = _mat(w, "w", (n, k), dt, dev)
    py, ldy = _mat(y, "y", out, yt, dev)
    pr, ldr = (None, n) if residual is None else _mat(residual, "residual", out, yt, dev)
    pz, ldz = (None, n) if z is None else _mat(z, "z", out, dt, dev)
    held, ws, nb = _scratch(ZERO_LINEAR, m, n, k, workspace, stream, x.device)
    _call(_lib.zero_linear, "zero_linear", dev, stream, px, _CODE[dt], ldx, pw, ldw,
          None if bias is None else _buf(bias, "bias", n, dt, x.device), m, n, k, act,
          None if drop is None else drop._c(x.device), pr, ldr, py, _CODE[yt], ldy, pz, ldz, ws,
          nb)


def zero_linear_dgrad(dy, w, dx, act: int = ZERO_ACT_NONE, z=None, drop=None, residual=None,
                      stream=None, workspace=None):
    """dx = residual + D(act'(z) * (dy w)): dy [m][n] and w [n][k] bf16 or
    fp16, dx [m][k] of that type or fp32, residual of dx's type (it may be dx
    itself).  act, z [m][k] and drop are those of the call that made this
    layer's input.  Workspace as for zero_linear."""
    dt = _in_type(dy, "dy")
    m, n = _shape(dy, "dy")
    k = _shape(w, "w")[1]
    dev, out, xt = dy.get_device(), (m, k), _out_type(dx, dt, "dx")
    py, lddy = _mat(dy, "dy", (m, n), dt, dev)
    pw, ldw = _mat(w, "w", (n, k), dt, dev)
    px, lddx = _mat(dx, "dx", out, xt, dev)
    pr, ldr = (None, k) if residual is None else _mat(residual, "residual", out, xt, dev)
    pz, ldz = (None, k) if z is None else _mat(z, "z", out, dt, dev)
    held, ws, nb = _scratch(ZERO_LINEAR_DGRAD, m, n, k, workspace, stream, dy.device)
    _call(_lib.zero_linear_dgrad, "zero_linear_dgrad", dev, stream, py, _CODE[dt], lddy, pw, ldw,
          m, n, k, act, pz, ldz, None if drop is None else drop._c(dy.device), pr, ldr, px,
          _CODE[xt], lddx, ws, nb)


def zero_linear_wgrad(dy, x, dw, db=None, accumulate: bool = False, stream=None, workspace=None):
    """dw (+)= dy^T x and db (+)= the column sums of dy: dy [m][n] and x
    [m][k] bf16 or fp16, dw [n][k] and db (n elements) of that type or fp32,
    usually places in a flat gradient row; accumulate adds to what they hold
    (a later micro-batch).  Workspace as for zero_linear."""
    dt = _in_type(dy, "dy")
    m, n = _shape(dy, "dy")
    k = _shape(x, "x")[1]
    dev, gt = dy.get_device(), _out_type(dw, dt, "dw")
    py, lddy = _mat(dy, "dy", (m, n), dt, dev)
    px, ldx = _mat(x, "x", (m, k), dt, dev)
    pg, lddw = _mat(dw, "dw", (n, k), gt, dev)
    held, ws, nb = _scratch(ZERO_LINEAR_WGRAD, m, n, k, workspace, stream, dy.device)
    _call(_lib.zero_linear_wgrad, "zero_linear_wgrad", dev, stream, py, _CODE[dt], lddy, px, ldx,
          m, n, k, pg, _CODE[gt], lddw,
          None if db is None else _buf(db, "db", n, gt, dy.device), int(bool(accumulate)), ws, nb)


def zero_dropout(x, y, drop, residual=None, stream=None):
    """y = residual + D(x) (2-D, bf16, fp16 or fp32; y may be x or residual
    itself).  The backward pass is the same call on the gradient."""
    shape, dt = _shape(x, "x"), x.dtype
    code = _CODE.get(dt)
    if code is None:
        raise TypeError(f"x: bfloat16, float16 or float32 expected, got {dt}")
    if drop is None:
        raise TypeError("drop: a ZeroDropout is required")
    dev = x.get_device()
    px, ldx = _mat(x, "x", shape, dt, dev)
    py, ldy = _mat(y, "y", shape, dt, dev)
    pr, ldr = (None, shape[1]) if residual is None else _mat(residual, "residual", shape, dt, dev)
    _call(_lib.zero_dropout, "zero_dropout", dev, stream, px, code, ldx, shape[0], shape[1],
          drop._c(x.device), pr, ldr, py, ldy)
