"""zero_linear, zero_linear_dgrad and zero_linear_wgrad against plain 64-bit
forms.  Whole numbers small enough that every fp32 sum is exact make the
sums' comparison bitwise whatever their order; normal numbers check the
epilogues within derived bounds.  Outputs lie in wider buffers whose other
elements must stay as they were."""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu

ACTS = {"none": zs.ZERO_ACT_NONE, "relu": zs.ZERO_ACT_RELU, "gelu": zs.ZERO_ACT_GELU,
        "gelu_tanh": zs.ZERO_ACT_GELU_TANH, "silu": zs.ZERO_ACT_SILU}
CANARY = -77.0


class Box:
    """A matrix inside a buffer of canaries: `lead` elements before it, rows
    `pad` elements longer than it."""

    def __init__(self, rows, cols, dtype, lead=0, pad=0, data=None):
        self.shape, ld = (rows, cols), cols + pad
        self.buf = torch.full((lead + rows * ld + 64,), CANARY, dtype=dtype, device="cuda")
        self.view = self.buf[lead:lead + rows * ld].view(rows, ld)[:, :cols]
        if data is not None:
            self.view.copy_(data)
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[lead:lead + rows * ld].view(rows, ld)[:, :cols] = False

    def untouched(self):
        assert bool((self.buf[self.mask] == CANARY).all()), "written outside the matrix"


def whole(rows, cols, seed, top=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-top, top + 1, (rows, cols), generator=g).double()


def normal(rows, cols, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, cols), generator=g, dtype=torch.float64) * scale


def product64(a, b):
    """a b^T in float64 on the GPU (small numbers: exact)"""
    return (a.cuda() @ b.cuda().t()).cpu()


# lengths 0 and 1, odd ones, one off the tiles, tiles, a divided contraction,
# few rows with long ones, many tiles
SIZES = [(1, 1, 1), (1, 64, 64), (1, 6400, 1600), (3, 5, 7), (2, 130, 63), (16, 48, 4096),
         (17, 33, 65), (64, 128, 64), (65, 129, 127), (128, 128, 128), (127, 255, 129),
         (100, 1, 300), (5, 300, 0), (256, 256, 64), (300, 700, 513), (31, 40, 8191),
         (4100, 2300, 72), (3333, 3001, 130), (9, 40000, 24), (4200, 4176, 72),
         (4200, 72, 4176), (72, 4200, 4176), (24, 100, 1300), (32, 2000, 200), (33, 90, 1000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("lead,pad", [(0, 0), (8, 8), (5, 3)])
def test_products_of_whole_numbers_are_exact(m, n, k, lead, pad, dtype):
    print(f"\n[linear] {m} x {n} x {k} lead {lead} pad {pad} {dtype}", flush=True)
    x, w, dy = whole(m, k, 1), whole(n, k, 2), whole(m, n, 3)
    bx, bw, bdy = Box(m, k, dtype, lead, pad, x), Box(n, k, dtype, lead, pad, w), \
        Box(m, n, dtype, lead, pad, dy)
    y, dx = Box(m, n, torch.float32, lead, pad), Box(m, k, torch.float32, lead, pad)
    dw, db = Box(n, k, torch.float32, lead, pad), Box(1, n, torch.float32, lead)
    zs.zero_linear(bx.view, bw.view, y.view)
    torch.cuda.synchronize()
    assert torch.equal(y.view.cpu().double(), product64(x, w))
    y.untouched()
    zs.zero_linear_dgrad(bdy.view, bw.view, dx.view)
    torch.cuda.synchronize()
    assert torch.equal(dx.view.cpu().double(), product64(dy, w.t().contiguous()))
    dx.untouched()
    if k == 0:
        return
    want, sums = product64(dy.t().contiguous(), x.t().contiguous()), dy.sum(0)
    for times in (1, 2):
        zs.zero_linear_wgrad(bdy.view, bx.view, dw.view, db=db.view[0], accumulate=times > 1)
        torch.cuda.synchronize()
        assert torch.equal(dw.view.cpu().double(), times * want)
        assert torch.equal(db.view[0].cpu().double(), times * sums)
        dw.untouched()
        db.untouched()


def test_no_rows():
    """m = 0: outputs of no rows are no-ops, the weight gradient is a sum of nothing"""
    w = torch.ones(8, 16, dtype=torch.bfloat16, device="cuda")
    x, y = w.new_empty(0, 16), w.new_empty(0, 8)
    zs.zero_linear(x, w, y)
    zs.zero_linear_dgrad(y, w, x)
    dw, db = torch.full((8, 16), 3.0, device="cuda"), torch.full((8,), 4.0, device="cuda")
    zs.zero_linear_wgrad(y, x, dw, db=db, accumulate=True)
    assert bool((dw == 3).all()) and bool((db == 4).all())
    zs.zero_linear_wgrad(y, x, dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def _forward(m, n, k, dtype, out, act, p, bias, res, lead=0, pad=0, seed=11, keep_z=True):
    print(f"\n[linear] {m} x {n} x {k} {dtype} -> {out} {act} p {p} bias {bias} res {res} "
          f"lead {lead} pad {pad}", flush=True)
    x = normal(m, k, seed).to(dtype).double()
    w = normal(n, k, seed + 1, 1 / math.sqrt(max(k, 1))).to(dtype).double()
    b = normal(1, n, seed + 2).to(dtype).double() if bias else torch.zeros(1, n).double()
    r = normal(m, n, seed + 3).to(out).double() if res else torch.zeros(m, n).double()
    y, z = Box(m, n, out, lead, pad), Box(m, n, dtype, lead, pad)
    drop = zs.ZeroDropout(p, seed=0x123456789ABCDEF, offset=seed, row0=7) if p else None
    zs.zero_linear(Box(m, k, dtype, lead, pad, x).view, Box(n, k, dtype, lead, pad, w).view,
                   y.view, bias=Box(1, n, dtype, lead, 0, b).view[0] if bias else None,
                   act=ACTS[act], drop=drop,
                   residual=Box(m, n, out, lead, pad, r).view if res else None,
                   z=z.view if keep_z else None)
    torch.cuda.synchronize()
    sz = product64(x, w) + b
    ez = ref.sum_err(k + 1, product64(x.abs(), w.abs()) + b.abs())
    a, slope, ea, _ = ref.act64(sz, act)
    err = ea + 1.2 * ez                     # no slope passes 1.2 in size
    if p:
        keep, scale = ref.keep(m, n, p, 0x123456789ABCDEF, seed, 7), ref.scale32(p)
        a, err = torch.where(keep, a * scale, 0.0), torch.where(keep, (err + a.abs() * ref.U) * scale, 0.0)
    ref.check(y.view, a + r, err + (a + r).abs() * ref.U, "y")
    y.untouched()
    if keep_z:
        ref.check(z.view, sz, ez, "z")
        z.untouched()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("m,n,k,lead,pad", [(1, 100, 72, 0, 0), (33, 200, 130, 0, 4),
                                            (40, 67, 1100, 3, 1), (300, 520, 192, 0, 0)])
def test_forward_epilogue(m, n, k, lead, pad, dtype, out, act):
    _forward(m, n, k, dtype, out, act, 0.25, True, True, lead, pad)


@pytest.mark.parametrize("p,bias,res,keep_z", [(0.0, False, False, False), (0.0, True, False, True),
                                               (0.5, False, False, False), (0.0, False, True, False)])
@pytest.mark.parametrize("m,n,k", [(1, 333, 500), (129, 260, 96), (20, 96, 2600)])
def test_forward_with_parts_left_out(m, n, k, p, bias, res, keep_z):
    _forward(m, n, k, torch.bfloat16, torch.bfloat16, "gelu", p, bias, res, keep_z=keep_z)


def _dgrad(m, n, k, dtype, out, act, p, res, lead=0, pad=0, seed=21):
    print(f"\n[dgrad] {m} x {n} x {k} {dtype} -> {out} {act} p {p} res {res} lead {lead} pad {pad}",
          flush=True)
    dy = normal(m, n, seed).to(dtype).double()
    w = normal(n, k, seed + 1, 1 / math.sqrt(n)).to(dtype).double()
    zin = normal(m, k, seed + 2, 2.0).to(dtype).double()
    r = normal(m, k, seed + 3).to(out).double() if res else torch.zeros(m, k).double()
    dx = Box(m, k, out, lead, pad)
    drop = zs.ZeroDropout(p, seed=99, offset=(1 << 64) - 3, row0=(1 << 32) - m,
                          step=torch.tensor([5], device="cuda")) if p else None
    zs.zero_linear_dgrad(Box(m, n, dtype, lead, pad, dy).view, Box(n, k, dtype, lead, pad, w).view,
                         dx.view, act=ACTS[act],
                         z=Box(m, k, dtype, lead, pad, zin).view if act != "none" else None,
                         drop=drop, residual=Box(m, k, out, lead, pad, r).view if res else None)
    torch.cuda.synchronize()
    wt = w.t().contiguous()
    g, eg = product64(dy, wt), ref.sum_err(n, product64(dy.abs(), wt.abs()))
    _, slope, _, es = ref.act64(zin, act)
    want, err = g * slope, eg * slope.abs() + g.abs() * es + eg * es + (g * slope).abs() * ref.U
    if p:
        keep, scale = ref.keep(m, k, p, 99, 2, (1 << 32) - m), ref.scale32(p)
        want, err = torch.where(keep, want * scale, 0.0), \
            torch.where(keep, (err + want.abs() * ref.U) * scale, 0.0)
    ref.check(dx.view, want + r, err + (want + r).abs() * ref.U, "dx")
    dx.untouched()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float32)])
@pytest.mark.parametrize("m,n,k,lead,pad", [(1, 100, 72, 0, 0), (33, 130, 200, 0, 4),
                                            (40, 1100, 67, 3, 1), (300, 192, 520, 0, 0)])
def test_dgrad_epilogue(m, n, k, lead, pad, dtype, out, act):
    _dgrad(m, n, k, dtype, out, act, 0.25, True, lead, pad)


@pytest.mark.parametrize("p,res", [(0.0, False), (0.5, False), (0.0, True)])
def test_dgrad_with_parts_left_out(p, res):
    _dgrad(70, 200, 300, torch.bfloat16, torch.bfloat16, "silu", p, res)
    _dgrad(20, 2600, 96, torch.bfloat16, torch.bfloat16, "none", p, res)


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.bfloat16),
                                        (torch.float16, torch.float16),
                                        (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("m,n,k,lead,pad", [(1, 40, 50, 0, 0), (77, 130, 264, 1, 3),
                                            (4000, 128, 136, 0, 8), (513, 600, 700, 0, 0)])
def test_wgrad_over_micro_batches(m, n, k, lead, pad, dtype, grad):
    print(f"\n[wgrad] {m} x {n} x {k} {dtype} -> {grad} lead {lead} pad {pad}", flush=True)
    dw, db = Box(n, k, grad, lead, pad), Box(1, n, grad, lead)
    want_w = want_b = None
    for step in range(3):
        dy, x = normal(m, n, 31 + step).to(dtype).double(), normal(m, k, 41 + step).to(dtype).double()
        old_w, old_b = dw.view.cpu().double(), db.view[0].cpu().double()
        zs.zero_linear_wgrad(Box(m, n, dtype, lead, pad, dy).view,
                             Box(m, k, dtype, lead, pad, x).view, dw.view, db=db.view[0],
                             accumulate=step > 0)
        torch.cuda.synchronize()
        dyt, xt = dy.t().contiguous(), x.t().contiguous()
        w, b = product64(dyt, xt), dy.sum(0)
        ew, eb = ref.sum_err(m, product64(dyt.abs(), xt.abs())), ref.sum_err(m, dy.abs().sum(0))
        if step:
            w, b = w + old_w, b + old_b
        ref.check(dw.view, w, ew + w.abs() * ref.U, "dw")
        ref.check(db.view[0], b, eb + b.abs() * ref.U, "db")
        dw.untouched()
        db.untouched()


def test_outputs_over_their_residual():
    """y in the place of its residual, with and without a divided contraction"""
    for m, n, k in [(300, 520, 192), (20, 96, 2600), (1, 100, 640)]:
        x = normal(m, k, 1).to(torch.bfloat16).cuda()
        w = normal(n, k, 2, 0.1).to(torch.bfloat16).cuda()
        r = normal(m, n, 3).to(torch.bfloat16).cuda()
        apart, inplace = torch.empty_like(r), r.clone()
        zs.zero_linear(x, w, apart, residual=r)
        zs.zero_linear(x, w, inplace, residual=inplace)
        assert torch.equal(apart, inplace)
        dy = normal(m, n, 4).to(torch.bfloat16).cuda()
        r = normal(m, k, 5).to(torch.bfloat16).cuda()
        apart, inplace = torch.empty_like(r), r.clone()
        zs.zero_linear_dgrad(dy, w, apart, residual=r)
        zs.zero_linear_dgrad(dy, w, inplace, residual=inplace)
        assert torch.equal(apart, inplace)


def test_nan_and_infinity_where_the_mask_drops():
    """a dropped element is 0 though its value is NaN or infinite; a NaN of
    one row of x reaches no other row"""
    m, n, k, p = 40, 70, 96, 0.5
    x = normal(m, k, 1).to(torch.bfloat16)
    x[3, 5], x[17, 0] = math.nan, math.inf
    w = normal(n, k, 2).to(torch.bfloat16)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    zs.zero_linear(x.cuda(), w.cuda(), y, drop=zs.ZeroDropout(p, seed=5))
    keep = ref.keep(m, n, p, 5, 0)
    y = y.cpu()
    assert bool((y[~keep] == 0).all())
    assert bool(torch.isnan(y[3][keep[3]]).all())
    assert not bool(torch.isfinite(y[17][keep[17]]).any())
    rest = torch.ones(m, dtype=torch.bool)
    rest[3] = rest[17] = False
    assert bool(torch.isfinite(y[rest]).all())


def test_slopes_at_the_ends():
    """act' at infinities, signed zeros and values whose squares overflow:
    finite, and its limits"""
    vals = [0.0, -0.0, math.inf, -math.inf, 1e30, -1e30, 3e38, -3e38, 1e-40, 90.0, -90.0]
    k = len(vals)
    z = torch.tensor([vals], dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, k, dtype=torch.bfloat16, device="cuda")
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        dx = torch.empty(1, k, device="cuda")
        zs.zero_linear_dgrad(dy, w, dx, act=ACTS[act], z=z)
        got = dx.cpu()[0]
        mid = 0.0 if act == "relu" else 0.5
        want = torch.tensor([mid if abs(v) < 1e-30 else float(v > 0) for v in vals])
        if act == "relu":
            want[8] = 1.0
        assert torch.allclose(got, want, atol=1e-5, rtol=0), (act, got)


def test_same_bits_on_every_run_and_on_any_stream():
    m, n, k = 70, 300, 5000
    x, w = normal(m, k, 1).to(torch.bfloat16).cuda(), normal(n, k, 2).to(torch.bfloat16).cuda()
    first = torch.empty(m, n, device="cuda")
    zs.zero_linear(x, w, first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for use in (None, side, side.cuda_stream):
        y = torch.zeros(m, n, device="cuda")
        torch.cuda.synchronize()
        zs.zero_linear(x, w, y, stream=use)
        torch.cuda.synchronize()
        assert torch.equal(y, first)


def test_gradients_agree_with_differences():
    """dx, dW and db of sum(c * y) against central differences of the 64-bit
    forward form along random directions.  The inputs are fp16; the bound is
    the outputs' own (fp32 sums of exact products) plus the differences' h^2
    term, both far below 1e-3 of the sizes met here."""
    m, n, k = 12, 20, 24
    x, w = normal(m, k, 1).half(), normal(n, k, 2, 0.3).half()
    b, c = normal(1, n, 3).half(), normal(m, n, 4).half()
    z = torch.empty(m, n, dtype=torch.float16, device="cuda")
    y = torch.empty(m, n, device="cuda")
    zs.zero_linear(x.cuda(), w.cuda(), y, bias=b[0].cuda(), act=zs.ZERO_ACT_SILU, z=z)
    # dz = c * silu'(z): the identity as the next layer's weight
    eye = torch.eye(n).half().cuda()
    dz = torch.empty(m, n, dtype=torch.float16, device="cuda")
    zs.zero_linear_dgrad(c.cuda(), eye, dz, act=zs.ZERO_ACT_SILU, z=z)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((m, k), (n, k), (n,)))
    zs.zero_linear_dgrad(dz, w.cuda(), dx)
    zs.zero_linear_wgrad(dz, x.cuda(), dw, db=db)

    def loss(x, w, b):
        v = x @ w.t() + b
        return float((c.double() * v * torch.sigmoid(v)).sum())

    x, w, b = x.double(), w.double(), b.double()
    h = 1e-5
    for which, got in ((0, dx), (1, dw), (2, db.view(1, -1))):
        for trial in range(4):
            base = [x, w, b]
            d = normal(*base[which].shape, 50 + trial)
            up, down = list(base), list(base)
            up[which], down[which] = base[which] + h * d, base[which] - h * d
            diff = (loss(*up) - loss(*down)) / (2 * h)
            mine = float((got.cpu().double() * d).sum())
            size = float((got.cpu().double() * d).abs().sum())
            # z and dz were rounded to fp16: 2^-11 of dz each, and dz moves by
            # at most |z| 2^-11 |silu''| |c| (|silu''| <= 0.5)
            assert abs(mine - diff) <= 6 * 2.0 ** -11 * size, (which, trial, mine, diff)


def test_offsets_past_32_bits():
    """rows 2^30 + 8 elements apart (the last starts past 2^32 bytes), read
    and written in place"""
    ld, m, n, k = (1 << 30) + 8, 4, 40, 72
    x, w = whole(m, k, 1), whole(n, k, 2)
    buf = torch.zeros((m - 1) * ld + 256, dtype=torch.bfloat16, device="cuda")
    bx = buf.as_strided((m, k), (ld, 1), 0)
    by = buf.as_strided((m, n), (ld, 1), 128)   # between the rows of x
    bx.copy_(x)
    bw = w.to(torch.bfloat16).cuda()
    want = product64(x, w).to(torch.bfloat16)
    with pytest.raises(zs.ZeroValueError):      # their spans overlap
        zs.zero_linear(bx, bw, by)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    zs.zero_linear(bx, bw, y)
    assert torch.equal(y.cpu(), want)
    big = torch.zeros((40 - 1) * (1 << 26) + 256, dtype=torch.bfloat16, device="cuda")
    xs = whole(40, k, 3)                         # the tile kernel's rows, 128 MiB apart
    far = big.as_strided((40, k), (1 << 26, 1), 0)
    far.copy_(xs)
    y2 = torch.empty(40, n, dtype=torch.float32, device="cuda")
    zs.zero_linear(far, bw, y2)
    assert torch.equal(y2.cpu().double(), product64(xs, w))
    dw = torch.empty(n, k, dtype=torch.float32, device="cuda")
    dy = whole(40, n, 4)
    zs.zero_linear_wgrad(dy.to(torch.bfloat16).cuda(), far, dw)
    assert torch.equal(dw.cpu().double(), product64(dy.t().contiguous(), xs.t().contiguous()))
    out = big.as_strided((40, n), (1 << 26, 1), 128)
    zs.zero_linear(xs.to(torch.bfloat16).cuda(), bw, out)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), product64(xs, w).to(torch.bfloat16).double())
    zs.zero_dropout(out, out, zs.ZeroDropout(0.5, 3))
    keep = ref.keep(40, n, 0.5, 3, 0)
    assert torch.equal(out.cpu() != 0, keep & (product64(xs, w).to(torch.bfloat16) != 0))


def test_calls_in_turn_share_a_workspace():
    """products with divided contractions one after another on one scratch"""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    shapes = [(40, 96, 5000), (64, 200, 3000), (33, 40, 8191), (40, 96, 5000)]
    outs = []
    for i, (m, n, k) in enumerate(shapes):
        assert 0 < zs.zero_linear_workspace_bytes(zs.ZERO_LINEAR, m, n, k) <= ws.numel()
        x, w = whole(m, k, i), whole(n, k, i + 9)
        y = torch.empty(m, n, device="cuda")
        zs.zero_linear(x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda(), y, workspace=ws)
        outs.append((y, product64(x, w)))
    torch.cuda.synchronize()
    for y, want in outs:
        assert torch.equal(y.cpu().double(), want)


def test_the_binding_refuses_before_a_launch():
    x, w = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((40, 64), (48, 64)))
    y = torch.full((40, 48), CANARY, dtype=torch.bfloat16, device="cuda")
    bad = [(TypeError, dict(y=y.to(torch.float16))), (ValueError, dict(y=y[:39])),
           (ValueError, dict(w=w[:, :60])), (TypeError, dict(w=w.half())),
           (TypeError, dict(w=torch.ones(64, 48, dtype=torch.bfloat16, device="cuda").t())),
           (TypeError, dict(x=x[0])), (TypeError, dict(x=x[:1].expand(40, 64))),
           (ValueError, dict(bias=w[0, :40])), (TypeError, dict(bias=w[0].float())),
           (ValueError, dict(residual=y[:, :40])), (TypeError, dict(residual=y.float())),
           (ValueError, dict(z=y[:3])), (ValueError, dict(act=9)),
           (ValueError, dict(drop=zs.ZeroDropout(1.0))),
           (TypeError, dict(drop=zs.ZeroDropout(0.1, step=torch.ones(1, device="cuda")))),
           (ValueError, dict(y=x.view(-1)[:40 * 48].view(40, 48)))]
    for err, change in bad:
        args = {**dict(x=x, w=w, y=y), **change}
        with pytest.raises(err):
            zs.zero_linear(args.pop("x"), args.pop("w"), args.pop("y"), **args)
    long = torch.ones(40, 8192, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        zs.zero_linear(long, long[:8], y[:, :8],
                       workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        zs.zero_linear_dgrad(y, w, x, act=zs.ZERO_ACT_SILU)
    torch.cuda.synchronize()
    assert bool((y == CANARY).all())


# undivided contractions without a mask, or with a mask and no activation: the
# straight epilogues, at sizes inside one tile, off the tiles and of the largest
STRAIGHT = [(70, 130, 64), (300, 520, 64), (129, 261, 50), (4104, 2600, 576)]


@pytest.mark.parametrize("act,p", [("gelu_tanh", 0.0), ("silu", 0.0), ("none", 0.25)])
@pytest.mark.parametrize("m,n,k", STRAIGHT)
def test_straight_forward_epilogues(m, n, k, act, p):
    assert zs.zero_linear_workspace_bytes(zs.ZERO_LINEAR, m, n, k) == 0
    big = m > 1000
    for dtype, out, bias, res, keep_z in (
            ((torch.bfloat16, torch.bfloat16, True, True, True),) if big else
            ((torch.bfloat16, torch.bfloat16, True, True, True),
             (torch.float16, torch.float16, False, False, False),
             (torch.bfloat16, torch.float32, True, True, False))):
        _forward(m, n, k, dtype, out, act, p, bias, res, keep_z=keep_z)


@pytest.mark.parametrize("act,p", [("gelu_tanh", 0.0), ("silu", 0.0), ("none", 0.25)])
@pytest.mark.parametrize("m,k,n", STRAIGHT)
def test_straight_dgrad_epilogues(m, n, k, act, p):
    assert zs.zero_linear_workspace_bytes(zs.ZERO_LINEAR_DGRAD, m, n, k) == 0
    _dgrad(m, n, k, torch.bfloat16, torch.bfloat16, act, p, True)
    if m < 1000:
        _dgrad(m, n, k, torch.float16, torch.float32, act, p, False)
