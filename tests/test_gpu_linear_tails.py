"""The activations and their slopes far out, where the falling side is many
orders below one: the error is held relative to the value itself, not to the
size of the sigmoid or of erf.  Products of one term (x 1) put every value of a
16-bit sweep through each epilogue."""
import math

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu

U = ref.U
ACTS = {"gelu": zs.ZERO_ACT_GELU, "gelu_tanh": zs.ZERO_ACT_GELU_TANH, "silu": zs.ZERO_ACT_SILU}
FLOOR = 2.0 ** -126   # exp2, the reciprocal and erfc may flush what is below


def _bounds(v, act):
    """act(v), act'(v) and how far their fp32 evaluation may be off.

    Sigmoid: s = 1 / (1 + e), e = 2^w.  w carries four roundings of its terms
    (6 |u| U at most with the folded constants'), e two units more, 1 + e and
    the reciprocal four: e's error moves s by s (1 - s) of it.  t = s - s^2 is
    one rounding and moves by at most as much as s.  erfc(x): 8 U its own, and
    its argument's two roundings times |x erfc'(x) / erfc(x)| <= 2 x^2 + 2 =
    v^2 + 2.  exp2(-v^2 / 2 log2 e): three roundings of the exponent, v^2 / 2
    each, and two units."""
    if act == "gelu":
        s = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        t, d = torch.exp(-v * v / 2), v / math.sqrt(2 * math.pi)
        es = s * (2 * (v * v + 2) + 10) * U + FLOOR
        et = t * (1.5 * v * v + 3) * U + FLOOR
    else:
        u = v if act == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
        s = torch.sigmoid(u)
        d = v if act == "silu" else v * math.sqrt(8 / math.pi) * (1 + 0.134145 * v * v)
        t = s * torch.sigmoid(-u)
        es = U * s * (torch.sigmoid(-u) * (6 * u.abs() + 4) + 4) + FLOOR
        et = es + U * t
    value, slope = v * s, s + t * d
    return value, slope, v.abs() * es + 2 * U * value.abs(), \
        es + d.abs() * et + 5 * U * (t * d).abs() + 2 * U * slope.abs()


def _sweep(dtype):
    """every sign and size from 2^-6 to 16 in steps of 1 / 64 of an octave"""
    e = torch.arange(-6 * 64, 4 * 64, dtype=torch.float64) / 64
    v = (2.0 ** e).to(dtype)
    return torch.cat([v, -v, torch.zeros(1, dtype=dtype)])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("rows,cols", [(1281, 16), (20, 7)])
def test_values(act, dtype, out, rows, cols):
    """many rows (tiles), few rows (their own kernel)"""
    v = _sweep(dtype)
    w = torch.ones(cols, 1, dtype=dtype, device="cuda")
    want, _, err, _ = _bounds(v.double(), act)
    for at in range(0, len(v), rows):
        x = v[at:at + rows].view(-1, 1).cuda()
        y = torch.empty(len(x), cols, dtype=out, device="cuda")
        zs.zero_linear(x, w, y, act=ACTS[act])
        part = slice(at, at + rows)
        ref.check(y, want[part, None].expand(-1, cols), err[part, None].expand(-1, cols), act)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_slopes(act, dtype, out, p):
    v = _sweep(dtype)
    rows, k = 3, len(v)
    z = v.expand(rows, -1).contiguous().cuda()
    dy = torch.ones(rows, 1, dtype=dtype, device="cuda")
    w = torch.ones(1, k, dtype=dtype, device="cuda")
    dx = torch.empty(rows, k, dtype=out, device="cuda")
    zs.zero_linear_dgrad(dy, w, dx, act=ACTS[act], z=z,
                         drop=zs.ZeroDropout(p, seed=3) if p else None)
    _, want, _, err = (t.expand(rows, -1) for t in _bounds(v.double(), act))
    if p:
        keep, scale = ref.keep(rows, k, p, 3, 0), ref.scale32(p)
        want, err = torch.where(keep, want * scale, 0.0), \
            torch.where(keep, err * scale + U * (want * scale).abs(), 0.0)
    ref.check(dx, want, err, act)
