"""The binding of include/zero_norm.h: the layer norm on the flat 16-bit
buffers.

    w, b = weights[o1:o1 + n], weights[o2:o2 + n]          # the all-gather buffer
    zero_layernorm(x, w, b, y, mean=mean, rstd=rstd)
    zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=d, dw=row[o1:o1 + n],
                            db=row[o2:o2 + n])

As for the layer products, matrices are 2-D tensors or views whose rows are
contiguous, everything is checked before a launch, and autograd records
nothing.
"""
import ctypes

import torch

from . import _lib
from ._linear import _CODE, _call, _in_type, _mat, _out_type, _scratch_of, _shape, _vec


def _declare(L):
    vp, i64, i32, enum = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    L.zero_layernorm.argtypes = [vp, enum, i64, vp, vp, enum, i64, i64, ctypes.c_double, vp, enum,
                                 i64, vp, vp, vp]
    L.zero_layernorm.restype = enum
    L.zero_layernorm_workspace_bytes.argtypes = [i64, i64]
    L.zero_layernorm_workspace_bytes.restype = i64
    L.zero_layernorm_backward.argtypes = [vp, enum, i64, vp, enum, i64, vp, enum, vp, vp, i64, i64,
                                          vp, i64, vp, i64, vp, vp, enum, i32, vp, i64, vp]
    L.zero_layernorm_backward.restype = enum


_declare(_lib)


def _weight_type(w, b, *others):
    """the 16-bit type of the flat buffer: the weight's, the bias's, or (with
    neither) that of the first other tensor that is not fp32"""
    for t, what in ((w, "w"), (b, "b")):
        if t is not None:
            return _in_type(t, what)
    for t in others:
        if t is not None and t.dtype in (torch.bfloat16, torch.float16):
            return t.dtype
    return torch.bfloat16


def zero_layernorm(x, w, b, y, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """y = (x - mean) rstd w + b over each row of x [m][n], rstd = 1 / sqrt(var
    + eps): w and b (n elements, bf16 or fp16) may be None, x and y are of
    their type or fp32 (y may be x itself); mean and rstd (fp32, m elements)
    are written for the backward pass where given."""
    m, n = _shape(x, "x")
    dt = _weight_type(w, b, x, y)
    xt, yt, dev = _out_type(x, dt, "x"), _out_type(y, dt, "y"), x.get_device()
    px, ldx = _mat(x, "x", (m, n), xt, dev)
    py, ldy = _mat(y, "y", (m, n), yt, dev)
    _call(_lib.zero_layernorm, "zero_layernorm", dev, stream, px, _CODE[xt], ldx,
          _vec(w, "w", n, dt, dev), _vec(b, "b", n, dt, dev), _CODE[dt], m, n, eps, py, _CODE[yt],
          ldy, _vec(mean, "mean", m, torch.float32, dev), _vec(rstd, "rstd", m, torch.float32, dev))


def zero_layernorm_workspace_bytes(m: int, n: int) -> int:
    """Bytes of device workspace the backward pass of m rows of n needs where
    dw or db is asked for."""
    b = _lib.zero_layernorm_workspace_bytes(m, n)
    if b < 0:
        raise ValueError(f"zero_layernorm_workspace_bytes: m {m}, n {n} out of range")
    return b


def zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=None, dw=None, db=None,
                            accumulate: bool = False, stream=None, workspace=None):
    """dx = residual + the gradient of zero_layernorm's x, and dw (+)=, db (+)=
    those of its weight and bias: x, mean and rstd as the forward call read
    and wrote them; dy of w's type or fp32, dx and residual of x's (dx may be
    residual or dy itself); dw and db (n elements of w's type or fp32, usually
    places in a flat gradient row) may be None, and accumulate adds to what
    they hold.  A workspace tensor is allocated where one is needed unless one
    of zero_layernorm_workspace_bytes(m, n) bytes is passed."""
    m, n = _shape(x, "x")
    dt = _weight_type(w, None, x, dy, dw, db)
    xt, yt, dev = _out_type(x, dt, "x"), _out_type(dy, dt, "dy"), x.get_device()
    gt = torch.float32 if dw is None and db is None else \
        _out_type(dw if dw is not None else db, dt, "dw" if dw is not None else "db")
    px, ldx = _mat(x, "x", (m, n), xt, dev)
    py, lddy = _mat(dy, "dy", (m, n), yt, dev)
    pd, lddx = _mat(dx, "dx", (m, n), xt, dev)
    pr, ldr = (None, n) if residual is None else _mat(residual, "residual", (m, n), xt, dev)
    need = 0 if workspace is not None or (dw is None and db is None) else \
        zero_layernorm_workspace_bytes(m, n)
    held, ws, nb = _scratch_of(need, workspace, stream, x.device)
    _call(_lib.zero_layernorm_backward, "zero_layernorm_backward", dev, stream, py, _CODE[yt],
          lddy, px, _CODE[xt], ldx, _vec(w, "w", n, dt, dev), _CODE[dt],
          _vec(mean, "mean", m, torch.float32, dev), _vec(rstd, "rstd", m, torch.float32, dev), m,
          n, pr, ldr, pd, lddx, _vec(dw, "dw", n, gt, dev), _vec(db, "db", n, gt, dev), _CODE[gt],
          int(bool(accumulate)), ws, nb)
