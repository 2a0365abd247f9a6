"""The binding of include/zero_muon.h: the Muon step of a shard.

    zero_muon_momentum(grads, n_dp, ld, length, mom, u, hp)      # this rank's range
    zero_orthogonalize(u[off:off + r * c].view(r, c), o[off:off + r * c].view(r, c))
    zero_muon_update(o[a:b], master, weights, layout, rank, hp, update_scale=k)

hp is the AdamWHParams of the rest of the step: lr, beta1 (the momentum),
weight_decay and grad_scale take part.  A stack of matrices of one shape, for
instance the same matrix of every layer, is one 3-D view of the flat buffer.
"""
import ctypes

import torch

from . import (ZeroValueError, ZERO_EINVAL, _consts, _dtype_code, _lib, _rows, _slot_end,
               _StepControl)
from ._linear import _CODE, _call, _in_type, _scratch_of, _vec

ZERO_NS_MAX_STEPS = 32


class _NsParams(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("reserved", ctypes.c_int32), ("eps", ctypes.c_double),
                ("coeffs", ctypes.c_void_p)]


def _declare(L):
    vp, i64, i32, enum = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    L.zero_muon_momentum.argtypes = [vp, enum, i32, i64, i64, vp, vp, enum, i32, vp, vp, vp]
    L.zero_muon_momentum.restype = enum
    L.zero_muon_momentum_dc.argtypes = L.zero_muon_momentum.argtypes
    L.zero_muon_momentum_dc.restype = enum
    L.zero_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64]
    L.zero_orthogonalize_workspace_bytes.restype = i64
    L.zero_orthogonalize.argtypes = [vp, enum, i64, i64, i64, i64, i64,
                                     ctypes.POINTER(_NsParams), vp, enum, i64, i64, vp, i64, vp]
    L.zero_orthogonalize.restype = enum
    L.zero_muon_update.argtypes = [vp, enum, vp, vp, enum, vp, i32, i64, i64, vp,
                                   ctypes.c_double, vp, vp]
    L.zero_muon_update.restype = enum
    L.zero_muon_update_dc.argtypes = L.zero_muon_update.argtypes
    L.zero_muon_update_dc.restype = enum


_declare(_lib)


def _code(t, what):
    """the type code of a bf16, fp16 or fp32 tensor"""
    code = _CODE.get(getattr(t, "dtype", None))
    return _dtype_code(t, what, True) if code is None else code


def _device(t, what):
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: a GPU tensor is required")
    return t.get_device()


def _momentum(fn, what, grads, n_rows, ld, length, mom, u, consts, nesterov, skip, sumsq, max_norm,
              loss_scale, stream):
    dev = _device(mom, "mom")
    ctl = None
    if skip is not None or sumsq is not None or loss_scale is not None:
        ctl = ctypes.byref(_StepControl(
            _vec(skip, "skip", 1, torch.int32, dev), _vec(sumsq, "sumsq", 1, torch.float64, dev),
            float(max_norm), _vec(loss_scale, "loss_scale", 2, torch.int32, dev)))
    gc, uc = _code(grads, "grads"), _code(u, "u")
    _call(fn, what, dev, stream, _rows(grads, "grads", n_rows, ld, length, device=mom.device), gc,
          n_rows, ld, length, _vec(mom, "mom", length, torch.float32, dev),
          _vec(u, "u", length, u.dtype, dev), uc, int(bool(nesterov)), consts, ctl)


def zero_muon_momentum(grads, n_rows: int, ld: int, length: int, mom, u, hp,
                       nesterov: bool = True, skip=None, sumsq=None, max_norm: float = 0.0,
                       loss_scale=None, stream=None):
    """mom = beta1 mom + g and u = g + beta1 mom (nesterov) or mom, g the sum
    of the n_rows rows of grads (ld elements apart; bf16, fp16 or fp32) times
    grad_scale: mom[:length] fp32, u[:length] bf16, fp16 or fp32.  skip, sumsq
    with max_norm, and loss_scale as for zero_shard_adamw_ex."""
    hpc = hp._c()
    _momentum(_lib.zero_muon_momentum, "zero_muon_momentum", grads, n_rows, ld, length, mom, u,
              ctypes.byref(hpc), nesterov, skip, sumsq, max_norm, loss_scale, stream)


def zero_muon_momentum_dc(grads, n_rows: int, ld: int, length: int, mom, u, consts,
                          nesterov: bool = True, skip=None, sumsq=None, max_norm: float = 0.0,
                          loss_scale=None, stream=None):
    """zero_muon_momentum with its constants read from the device buffer
    consts when the kernel runs."""
    _momentum(_lib.zero_muon_momentum_dc, "zero_muon_momentum_dc", grads, n_rows, ld, length, mom,
              u, _consts(consts, mom.device), nesterov, skip, sumsq, max_norm, loss_scale, stream)


def zero_orthogonalize_workspace_bytes(count: int, rows: int, cols: int) -> int:
    """Bytes of device workspace zero_orthogonalize needs for count matrices
    of rows x cols."""
    b = _lib.zero_orthogonalize_workspace_bytes(count, rows, cols)
    if b < 0:
        raise ValueError(f"zero_orthogonalize_workspace_bytes: count {count}, rows {rows}, "
                         f"cols {cols} out of range")
    return b


def _stack(t, what, shape, dtypes, dev):
    """(address, row stride, matrix stride) of a 2-D matrix or a 3-D stack of
    them whose rows are contiguous and in order"""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{what}: a GPU tensor is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: one of {', '.join(map(str, dtypes))} expected, got {t.dtype}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, the call's tensors are on cuda:{dev}")
    if t.dim() not in (2, 3):
        raise TypeError(f"{what}: a 2-D or 3-D tensor is required, got {t.dim()}-D")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: {tuple(shape)} expected, got {tuple(t.shape)}")
    r, c = t.shape[-2:]
    s0, s1 = t.stride()[-2:]
    if c > 1 and s1 != 1:
        raise TypeError(f"{what}: rows of contiguous elements are required")
    if r > 1 and s0 < c:
        raise TypeError(f"{what}: rows that do not overlap are required (row stride {s0})")
    ld = s0 if r > 1 else max(c, 1)
    span = (r - 1) * ld + c if r and c else 0
    stride = t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else span
    if stride < span:
        raise TypeError(f"{what}: matrices that do not overlap are required (stride {stride})")
    return t.data_ptr(), ld, stride


def zero_orthogonalize(u, o, steps: int = 5, coeffs=None, eps: float = 1e-7, stream=None,
                       workspace=None):
    """o = u / (|u| + eps) after `steps` Newton-Schulz rounds, for a matrix
    [rows][cols] or a stack [count][rows][cols] (bf16, fp16 or fp32; o of the
    same shape, bf16 or fp16, any strides whose rows are contiguous).  coeffs:
    one (a, b, c) for each round, or None for (3.4445, -4.7750, 2.0315).  A
    workspace tensor is allocated unless one of
    zero_orthogonalize_workspace_bytes(count, rows, cols) bytes is passed."""
    pu, ldu, su = _stack(u, "u", None, (torch.bfloat16, torch.float16, torch.float32), None)
    dev = u.get_device()
    po, ldo, so = _stack(o, "o", u.shape, (torch.bfloat16, torch.float16), dev)
    rows, cols = u.shape[-2:]
    count = u.shape[0] if u.dim() == 3 else 1
    flat = None
    if coeffs is not None:
        flat = [float(v) for abc in coeffs for v in abc]
        if len(flat) != 3 * steps or any(len(abc) != 3 for abc in coeffs):
            raise ValueError(f"coeffs: one (a, b, c) for each of the {steps} rounds expected")
        if steps > ZERO_NS_MAX_STEPS:
            raise ZeroValueError(ZERO_EINVAL, "zero_orthogonalize")
        flat = (ctypes.c_double * len(flat))(*flat)
    ns = _NsParams(steps, 0, eps, None if flat is None else ctypes.addressof(flat))
    need = 0 if workspace is not None else \
        _lib.zero_orthogonalize_workspace_bytes(count, rows, cols)
    held, ws, nb = _scratch_of(need, workspace, stream, u.device)
    _call(_lib.zero_orthogonalize, "zero_orthogonalize", dev, stream, pu, _CODE[u.dtype], ldu, su,
          count, rows, cols, ctypes.byref(ns), po, _CODE[o.dtype], ldo, so, ws, nb)


def _update(fn, what, o, master, weight_full, layout, rank, consts, update_scale, shard_off,
            length, skip, stream):
    dev = _device(master, "master")
    if length is None:
        length = master.numel()
    ot, wt = _in_type(o, "o"), _in_type(weight_full, "weight_full")
    _call(fn, what, dev, stream, _vec(o, "o", length, ot, dev), _CODE[ot],
          _vec(master, "master", length, torch.float32, dev),
          _vec(weight_full, "weight_full", _slot_end(layout, rank, shard_off, length), wt, dev),
          _CODE[wt], ctypes.byref(layout), rank, shard_off, length, consts, update_scale,
          _vec(skip, "skip", 1, torch.int32, dev))


def zero_muon_update(o, master, weight_full, layout, rank: int, hp, update_scale: float = 1.0,
                     shard_off: int = 0, length=None, skip=None, stream=None):
    """master = master (1 - lr weight_decay) - lr (update_scale o) over
    [:length], cast into the shard's slot of weight_full (bf16 or fp16): o
    bf16 or fp16, the range's part of zero_orthogonalize's result."""
    hpc = hp._c()
    _update(_lib.zero_muon_update, "zero_muon_update", o, master, weight_full, layout, rank,
            ctypes.byref(hpc), update_scale, shard_off, length, skip, stream)


def zero_muon_update_dc(o, master, weight_full, layout, rank: int, consts,
                        update_scale: float = 1.0, shard_off: int = 0, length=None, skip=None,
                        stream=None):
    """zero_muon_update with lr and the decay read from the device buffer
    consts when the kernel runs."""
    _update(_lib.zero_muon_update_dc, "zero_muon_update_dc", o, master, weight_full, layout, rank,
            _consts(consts, master.device), update_scale, shard_off, length, skip, stream)
