"""Plain 64-bit forms of the layer products and the dropout, and the bounds
their tests use (written from the formulas; nothing here calls the library).

Rounding: a value stored in type t is off by at most half a step,
finfo(t).eps / 2 of itself (fp32 arithmetic: U = 2^-24), plus half the
smallest subnormal."""
import math

import numpy as np
import torch

U = 2.0 ** -24


def philox(c, key, rounds=10):
    """Philox4x32 of four uint64 arrays of 32-bit values under (k0, k1)"""
    s32, mask = np.uint64(32), np.uint64(0xFFFFFFFF)
    k0, k1 = key
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> s32) ^ c[1] ^ np.uint64(k0), p1 & mask,
             (p0 >> s32) ^ c[3] ^ np.uint64(k1), p0 & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def bits16(rows, cols, seed, stream, row0=0):
    """the 16 random bits of every element, [rows][cols]"""
    col = np.arange(cols)
    block = (col // 32 * 4 + col % 16 // 4).astype(np.uint64)[None, :]
    zero = np.zeros((rows, cols), np.uint64)
    row = (np.arange(rows, dtype=np.uint64) + np.uint64(row0))[:, None]
    stream &= (1 << 64) - 1
    w = philox([zero + block, zero + row, zero + np.uint64(stream & 0xFFFFFFFF),
                zero + np.uint64(stream >> 32)], (seed & 0xFFFFFFFF, seed >> 32))
    pick = np.choose(np.broadcast_to(col % 4, (rows, cols)), w)
    return ((pick >> (16 * (col % 32 // 16)).astype(np.uint64)) & np.uint64(0xFFFF)).astype(np.int64)


def threshold(p):
    return min(65535, int(np.rint(p * 65536)))


def keep(rows, cols, p, seed, stream, row0=0):
    return torch.from_numpy(bits16(rows, cols, seed, stream, row0) >= threshold(p))


def scale32(p):
    """the factor of a kept element, as fp32 rounds it"""
    return float(np.float32(65536.0 / (65536 - threshold(p))))


def act64(v, name):
    """act(v), act'(v) and the bounds (relative to |v| and absolute) of their
    fp32 evaluation, all float64.  A sigmoid of u carries the rounding of u
    (six roundings of its terms, |u| each) and of exp2, 1 + e and the
    reciprocal (eight units in all): es = s (6 |u| + 8) U."""
    zero = torch.zeros_like(v)
    if name == "none":
        return v, zero + 1, zero, zero
    if name == "relu":
        return torch.where(v > 0, v, zero), (v > 0).double(), zero, zero
    if name == "gelu":
        s = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        t, d = torch.exp(-v * v / 2), v / math.sqrt(2 * math.pi)
        # erff to 2 units, 1 + erf and the products to one each
        es = zero + 4 * U
        et = t * (6 * v * v + 8) * U
    else:
        u = v if name == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
        s = torch.sigmoid(u)
        d = v if name == "silu" else v * math.sqrt(8 / math.pi) * (1 + 0.134145 * v * v)
        t = s * torch.sigmoid(-u)
        es = s * (6 * u.abs() + 8) * U
        et = es + 2 * U
    return v * s, s + t * d, v.abs() * (es + 2 * U * s), es + d.abs() * et + 6 * U * (t * d).abs() + 2 * U


def stored(ref, err, dtype):
    """the bound of an output within err of ref and then rounded to dtype"""
    f = torch.finfo(dtype)
    return err + (ref.abs() + err) * (f.eps / 2) + f.smallest_normal * f.eps


def check(got, ref, err, what):
    """|got - ref| <= the bound everywhere"""
    got, ref = got.detach().cpu(), ref.cpu()
    tol = stored(ref, err.cpu(), got.dtype)
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst " \
        f"{float((off / tol).nan_to_num(nan=math.inf).max()):.3g} of the bound"


def sum_err(k, mag):
    """bound of a k-term fp32 sum whose terms' magnitudes add up to mag: one
    rounding (of at most a whole unit, 2 U) a term, in any order"""
    return (k + 2) * 2 * U * mag
