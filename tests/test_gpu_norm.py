"""The layer norm against its formulas in 64 bits, on the GPU.

Tolerances.  u = 2^-24 is fp32's half step.  A sum of n fp32 terms, added eight
at a time per lane and then over lanes and waves in a tree, is off by at most
(8 K + 24) u times the sum of the magnitudes (K <= 4 pieces a lane; rows read
in a loop: 8 + n / 8192 + 24); SUM below covers both up to n = 300,000.  mean0
has that error, but s1 / n, the mean of the differences, takes it back to the
differences' own SUM u |d|.  So (x - mean) is off by SUM u times the row's mean
absolute difference, at most SUM u / rstd, rstd by (SUM + 4) u relative, and y
by (2 SUM + 8) u (|h| + 1) |w| + 2 u |y| and its own rounding."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 72
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def rounding(t, v):
    """the most that rounding values of at most v to t can be off: half a step,
    eps / 2 of the value, and below the smallest normal number (fp16's 2^-14 is
    met here) half of the constant step eps x that number: 2^-25"""
    f = torch.finfo(t)
    return f.eps / 2 * v.clamp(min=f.smallest_normal)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, m, n, pad, t, scale=1.0, off=0, shift=0.0):
    """[m][n] of rows n + pad apart from element off of a buffer, and the buffer"""
    buf = (torch.randn(off + m * (n + pad) + 1, generator=g, device="cuda") * scale + shift).to(t)
    return buf[off:off + m * (n + pad)].view(m, n + pad)[:, :n], buf


def near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0].item()} for {want[bad][0].item()}, tolerance {tol[bad][0].item():.3g}"


def forward64(x, w, b, eps=EPS):
    x = x.double()
    d = x - x.mean(1, keepdim=True)
    rstd = ((d * d).mean(1, keepdim=True) + eps).rsqrt()
    h = d * rstd
    y = h * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return x.mean(1), rstd[:, 0], h, y


def check_forward(x, w, b, y, mean, rstd):
    m64, r64, h, y64 = forward64(x, w, b)
    aw = torch.ones((), device="cuda") if w is None else w.double().abs()
    tol = (2 * SUM + 8) * U * (h.abs() + 1) * aw + 2 * U * y64.abs()
    near(y, y64, tol + rounding(y.dtype, y64.abs() + tol), "y")
    if mean is not None:
        near(mean, m64, (SUM + 4) * U / r64 + 2 * U * m64.abs(), "mean")
    if rstd is not None:
        near(rstd, r64, (SUM + 4) * U * r64, "rstd")


# every way through: rows in a fraction of a wave, in one, in several, in a
# loop (below eight, beyond 16384), odd and even, few and many
SHAPES = [(1, 1), (5, 7), (3, 8), (70, 9), (33, 64), (100, 127), (4100, 128), (65, 129), (9, 255),
          (2100, 256), (40, 257), (1, 1600), (700, 1600), (515, 2001), (64, 4096), (3000, 4096),
          (600, 6401), (513, 8200), (520, 11008), (514, 13000), (3, 16384), (7, 16385),
          (2, 100001)]


@pytest.mark.parametrize("m,n", SHAPES)
def test_forward_over_sizes(m, n):
    g = gen(m * 7 + n)
    x, _ = rows(g, m, n, 3, BF)
    w, b = (torch.randn(n + 1, generator=g, device="cuda").to(BF)[1:] for _ in range(2))
    y, ybuf = rows(g, m, n, 5, BF)
    before = ybuf.clone()
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    zs.zero_layernorm(x, w, b, y, eps=EPS, mean=mean, rstd=rstd)
    check_forward(x, w, b, y, mean, rstd)
    y.copy_(before[:m * (n + 5)].view(m, n + 5)[:, :n])
    assert torch.equal(ybuf, before)  # nothing between the rows was written


@pytest.mark.parametrize("wt", [BF, HF])
@pytest.mark.parametrize("xf,yf", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("affine", ["wb", "w", "b", ""])
def test_forward_over_types(wt, xf, yf, affine):
    g = gen(3)
    for m, n in ((37, 100), (600, 1603), (3, 6400)):
        x, _ = rows(g, m, n, 1, F if xf else wt, off=1, shift=0.5)
        w = torch.randn(n, generator=g, device="cuda").to(wt) if "w" in affine else None
        b = torch.randn(n, generator=g, device="cuda").to(wt) if "b" in affine else None
        y, _ = rows(g, m, n, 0, F if yf else wt, off=1)
        zs.zero_layernorm(x, w, b, y, eps=EPS)
        check_forward(x, w, b, y, None, None)


def test_a_mean_far_from_zero_keeps_the_differences():
    # x = 1000 + d with d in sixteenths: the variance from sums of squares
    # would have no correct digit
    x = 1000.0 + torch.randint(-8, 9, (600, 1600), device="cuda", generator=gen(1)) / 16
    y, mean, rstd = torch.empty_like(x), torch.empty(600, device="cuda"), \
        torch.empty(600, device="cuda")
    w = torch.ones(1600, dtype=BF, device="cuda")
    zs.zero_layernorm(x, w, None, y, eps=EPS, mean=mean, rstd=rstd)
    check_forward(x, w, None, y, mean, rstd)


def test_forward_special_rows():
    g = gen(5)
    x = torch.randn(8, 1600, generator=g, device="cuda")
    x[1, 5], x[2, 1599], x[3, 0] = float("inf"), float("nan"), float("-inf")
    x[4] = 3.25
    x[5] = 0.0
    w = torch.randn(1600, generator=g, device="cuda").to(BF)
    y, mean, rstd = torch.empty(8, 1600, device="cuda"), torch.empty(8, device="cuda"), \
        torch.empty(8, device="cuda")
    zs.zero_layernorm(x, w, None, y, eps=EPS, mean=mean, rstd=rstd)
    assert y[1:4].isnan().all() and not y[[0, 4, 5, 6, 7]].isnan().any()
    assert mean[1] == float("inf") and mean[3] == float("-inf") and mean[2].isnan()
    assert rstd[1:4].isnan().all()
    assert (y[4:6] == 0).all() and mean[4] == 3.25  # constant rows: exact zeros
    keep = [0, 4, 5, 6, 7]
    check_forward(x[keep], w, None, y[keep], mean[keep], rstd[keep])


def test_forward_in_place():
    g = gen(6)
    for t, n in ((BF, 1600), (F, 2001), (HF, 20000)):
        x, _ = rows(g, 9, n, 4, t)
        w = torch.randn(n, generator=g, device="cuda").to(HF if t == HF else BF)
        want = torch.empty(9, n, dtype=t, device="cuda")
        zs.zero_layernorm(x, w, w, want)
        zs.zero_layernorm(x, w, w, x)
        assert torch.equal(x, want)


# ---------------------------------------------------------------------------
# backward: mean and rstd are inputs.  h and g are off by 3 u relative; the
# sums by SUM u of their magnitudes; dx by what they give, times rstd.  A
# column's sum runs over the rows of a lane, then of a workgroup, then over the
# workgroups: at most m / 128 + 8 + 32 + 16 additions in a row.


def check_backward(dy, x, w, mean, rstd, res, dx, dw, db, old=None):
    m, n = x.shape
    dy64, x64, r = dy.double(), x.double(), rstd.double()[:, None]
    w64 = torch.ones(n, dtype=torch.float64, device="cuda") if w is None else w.double()
    h = (x64 - mean.double()[:, None]) * r
    g = dy64 * w64
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    want = r * (g - c1 - h * c2)
    tol = U * r * (8 * g.abs() + (SUM + 8) * a1 + (SUM + 12) * h.abs() * a2)
    if res is not None:
        want = want + res.double()
        tol = tol + U * (want.abs() + res.double().abs())
    near(dx, want, tol + rounding(dx.dtype, want.abs() + tol), "dx")
    adds = m / 128 + 64
    for got, terms, first in ((dw, dy64 * h, 0), (db, dy64, 1)):
        if got is None:
            continue
        want, tol = terms.sum(0), (adds + 4) * U * terms.abs().sum(0)
        if old is not None:
            want = want + old[first].double()
            tol = tol + U * want.abs()
        near(got, want, tol + rounding(got.dtype, want.abs() + tol), "db" if first else "dw")


def backward_case(g, m, n, t, xt, yt, gt, residual, pad=3, weight=True):
    x, _ = rows(g, m, n, pad, xt, off=1, shift=0.25)
    dy, _ = rows(g, m, n, pad + 1, yt)
    w = torch.randn(n + 1, generator=g, device="cuda").to(t)[1:] if weight else None
    m64, r64, _, _ = forward64(x, None, None)
    mean, rstd = m64.float(), r64.float()
    res = rows(g, m, n, pad, xt)[0] if residual else None
    dx, dxbuf = rows(g, m, n, pad + 2, xt)
    row = torch.randn(2 * n + 3, generator=g, device="cuda").to(gt)
    return dy, x, w, mean, rstd, res, dx, dxbuf, row[1:1 + n], row[n + 2:2 * n + 2], row


@pytest.mark.parametrize("m,n", SHAPES + [(20000, 1600), (5000, 3000), (300, 20000)])
def test_backward_over_sizes(m, n):
    dy, x, w, mean, rstd, res, dx, dxbuf, dw, db, row = \
        backward_case(gen(m + 3 * n), m, n, BF, BF, BF, F, True)
    before, canaries = dxbuf.clone(), (row[0].item(), row[n + 1].item(), row[-1].item())
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
    check_backward(dy, x, w, mean, rstd, res, dx, dw, db)
    assert canaries == (row[0].item(), row[n + 1].item(), row[-1].item())
    dx.copy_(before[:m * (n + 5)].view(m, n + 5)[:, :n])
    assert torch.equal(dxbuf, before)
    first = dw.clone(), db.clone()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
    assert torch.equal(first[0], dw) and torch.equal(first[1], db)  # the same bits
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db,
                               accumulate=True)
    check_backward(dy, x, w, mean, rstd, res, dx, dw, db, old=first)


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("xf,yf,gf", [(False, False, False), (False, True, True),
                                      (True, False, True), (True, True, False)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_over_types(t, xf, yf, gf, residual):
    g = gen(11)
    for m, n in ((37, 100), (600, 1603), (900, 4096), (70, 9000), (30, 14000)):
        dy, x, w, mean, rstd, res, dx, _, dw, db, _ = backward_case(
            g, m, n, t, F if xf else t, F if yf else t, F if gf else t, residual)
        zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
        check_backward(dy, x, w, mean, rstd, res, dx, dw, db)


@pytest.mark.parametrize("n", [513, 2200, 3584, 3700, 4104, 5555, 8185, 8192, 8193, 12300])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F, F), (BF, F)])
def test_backward_of_each_split(n, xt, yt):
    """rows of 2 to 16 waves and of more than a piece a lane, some of them idle at the end"""
    for m in (300, 2100):
        dy, x, w, mean, rstd, res, dx, dxbuf, dw, db, row = \
            backward_case(gen(n + m), m, n, BF, xt, yt, F, m == 300)
        zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
        check_backward(dy, x, w, mean, rstd, res, dx, dw, db)


@pytest.mark.parametrize("m,n", [(8192, 4096), (8195, 3700), (8191, 4096), (6200, 1100),
                                 (4099, 2304), (16400, 600)])
@pytest.mark.parametrize("yt", [BF, F])
def test_backward_of_many_rows(m, n, yt):
    """one workgroup or two on a CU, one piece a lane or two"""
    dy, x, w, mean, rstd, res, dx, dxbuf, dw, db, row = \
        backward_case(gen(n + m), m, n, BF, BF, yt, F, True)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
    check_backward(dy, x, w, mean, rstd, res, dx, dw, db)
    part = dx.clone()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res)
    assert torch.equal(part, dx)


@pytest.mark.parametrize("m", [1, 7, 64, 511, 512, 513])
@pytest.mark.parametrize("n", [8, 129, 1601, 5000, 9001, 16384])
@pytest.mark.parametrize("gt", [BF, F])
def test_backward_of_few_rows(m, n, gt):
    """dx and the column sums by different workgroups; in place by one kind after the other"""
    dy, x, w, mean, rstd, res, dx, dxbuf, dw, db, row = \
        backward_case(gen(n + m), m, n, BF, BF, BF, gt, True)
    canaries = row[0].item(), row[n + 1].item(), row[-1].item()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
    check_backward(dy, x, w, mean, rstd, res, dx, dw, db)
    first = dw.clone(), db.clone()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, accumulate=True)
    assert torch.equal(db, first[1])
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, db=db, accumulate=True)
    check_backward(dy, x, w, mean, rstd, res, dx, dw, db, old=first)
    assert canaries == (row[0].item(), row[n + 1].item(), row[-1].item())
    kept = dy.clone()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dy, residual=dy, dw=dw, db=db)
    check_backward(kept, x, w, mean, rstd, kept, dy, dw, db)


@pytest.mark.parametrize("n", [513, 2200, 4097, 5000, 7000, 8192, 11000])
@pytest.mark.parametrize("xf,yf", [(True, True), (True, False), (False, True)])
def test_forward_of_each_split(n, xf, yf):
    g = gen(n)
    for m in (513, 4099):
        x, _ = rows(g, m, n, 1, F if xf else BF, off=1, shift=0.5)
        w, b = (torch.randn(n, generator=g, device="cuda").to(BF) for _ in range(2))
        y, _ = rows(g, m, n, 0, F if yf else BF, off=1)
        zs.zero_layernorm(x, w, b, y, eps=EPS)
        check_forward(x, w, b, y, None, None)


@pytest.mark.parametrize("n", [100, 1600, 20000])
def test_backward_without_some_gradients(n):
    dy, x, _, mean, rstd, res, dx, _, dw, db, row = \
        backward_case(gen(2), 50, n, BF, BF, BF, BF, False, weight=False)
    kept = row.clone()
    zs.zero_layernorm_backward(dy, x, None, mean, rstd, dx)
    check_backward(dy, x, None, mean, rstd, None, dx, None, None)
    assert torch.equal(row, kept)
    zs.zero_layernorm_backward(dy, x, None, mean, rstd, dx, db=db)
    check_backward(dy, x, None, mean, rstd, None, dx, None, db)
    assert torch.equal(dw, kept[1:1 + n])
    zs.zero_layernorm_backward(dy, x, None, mean, rstd, dx, dw=dw)
    check_backward(dy, x, None, mean, rstd, None, dx, dw, db)


@pytest.mark.parametrize("n", [100, 1600, 6401, 20000])
def test_backward_in_place(n):
    g = gen(8)
    dy, x, w, mean, rstd, res, dx, _, dw, db, _ = backward_case(g, 600, n, BF, BF, BF, F, True)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db)
    want = dx.clone(), dw.clone(), db.clone()
    r2 = res.clone()
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, r2, residual=r2, dw=dw, db=db)
    assert torch.equal(r2, want[0])
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dy, residual=res, dw=dw, db=db)
    assert torch.equal(dy, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])


def test_no_rows_give_zero_sums():
    x = torch.empty(0, 100, dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    dw, db = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    zs.zero_layernorm(x, None, None, x, mean=s, rstd=s)
    zs.zero_layernorm_backward(x, x, None, s, s, torch.empty_like(x), dw=dw, db=db,
                               accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    zs.zero_layernorm_backward(x, x, None, s, s, torch.empty_like(x), dw=dw, db=db)
    assert (dw == 0).all() and (db == 0).all()


def test_gradients_against_differences():
    """of sum(c y) in x, w and b, in fp32; central differences of the 64-bit
    formula at 2^-10, whose own error is of the order of 2^-20"""
    g = gen(4)
    m, n = 6, 50
    x, c = (torch.randn(m, n, generator=g, device="cuda") for _ in range(2))
    w, b = (torch.randn(n, generator=g, device="cuda").to(BF) for _ in range(2))
    y, mean, rstd = torch.empty_like(x), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    zs.zero_layernorm(x, w, b, y, eps=EPS, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    zs.zero_layernorm_backward(c, x, w, mean, rstd, dx, dw=dw, db=db)
    x64, w64, b64, c64 = x.double(), w.double(), b.double(), c.double()

    def loss(x, w, b):
        return (c64 * forward64(x, w, b)[3]).sum()

    e = 2.0 ** -10
    for t, got in ((x64, dx), (w64, dw), (b64, db)):
        for i in range(0, t.numel(), 7):
            f = t.view(-1)
            v = f[i].item()
            f[i] = v + e
            up = loss(x64, w64, b64)
            f[i] = v - e
            down = loss(x64, w64, b64)
            f[i] = v
            assert abs((up - down).item() / (2 * e) - got.view(-1)[i].item()) < 2e-4


def test_other_streams_and_graphs():
    """a side stream; two graphs that share a workspace, replayed in turn with
    eager work of their own between"""
    g = gen(9)
    m, n = 700, 1601
    dy, x, w, mean, rstd, res, dx, _, dw, db, _ = backward_case(g, m, n, BF, BF, BF, F, True)
    b = torch.randn(n, generator=g, device="cuda").to(BF)
    y = torch.empty(m, n, dtype=BF, device="cuda")
    ws = torch.empty(zs.zero_layernorm_workspace_bytes(m, n), dtype=torch.uint8, device="cuda")

    def step():
        zs.zero_layernorm(x, w, b, y, mean=mean, rstd=rstd)
        zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db,
                                   workspace=ws)
        return [t.clone() for t in (y, mean, rstd, dx, dw, db)]

    outs = (y, mean, rstd, dx, dw, db)
    side = torch.cuda.Stream()
    want = step()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for t, v in zip(outs, want):
        assert torch.equal(t, v)
    zs.zero_layernorm(x, w, b, y, stream=side)  # a stream given by hand
    side.synchronize()
    assert torch.equal(y, want[0])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            zs.zero_layernorm(x, w, b, y, mean=mean, rstd=rstd)
            zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, residual=res, dw=dw, db=db,
                                       workspace=ws)
        graphs.append(graph)
    for k in range(4):
        x.copy_(torch.randn(m, n, generator=g, device="cuda"))
        dy.copy_(torch.randn(m, n, generator=g, device="cuda"))
        want = step()
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graphs[k & 1].replay()
        torch.cuda.synchronize()
        for t, v in zip(outs, want):
            assert torch.equal(t, v)


def test_the_binding_refuses_what_does_not_fit():
    x = torch.zeros(6, 32, dtype=BF, device="cuda")
    w = torch.zeros(32, dtype=BF, device="cuda")
    s = torch.zeros(6, device="cuda")
    y = torch.zeros_like(x)
    for bad in (dict(w=w[:31]), dict(w=w.float()), dict(b=w.half()), dict(y=y[:, :31]),
                dict(y=y.half()), dict(mean=s[:5]), dict(rstd=s.double()), dict(x=x.half()),
                dict(y=y.t().contiguous().t()), dict(eps=0.0)):
        with pytest.raises((TypeError, ValueError)):
            zs.zero_layernorm(**{**dict(x=x, w=w, b=w, y=y), **bad})
    ok = dict(dy=y, x=x, w=w, mean=s, rstd=s, dx=torch.zeros_like(x), dw=w.float(), db=w.float())
    for bad in (dict(dy=y[:5]), dict(dx=x.float()), dict(dw=w), dict(db=w.float()[:31]),
                dict(residual=x.float()), dict(mean=None), dict(dx=x),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            zs.zero_layernorm_backward(**{**ok, **bad})


def test_more_elements_than_32_bits_count():
    """rows behind element 2^31 of x and y"""
    m, n = 530000, 4096
    x = torch.zeros(m, n, dtype=BF, device="cuda")
    x[-600:] = torch.randn(600, n, generator=gen(3), device="cuda").to(BF)
    w = torch.randn(n, generator=gen(4), device="cuda").to(BF)
    y, mean, rstd = torch.empty_like(x), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    zs.zero_layernorm(x, w, None, y, mean=mean, rstd=rstd)
    check_forward(x[-600:], w, None, y[-600:], mean[-600:], rstd[-600:])
    assert (y[:1000] == 0).all() and (y[-1000:-600] == 0).all()
    dx, db = torch.empty_like(x), torch.empty(n, device="cuda")
    zs.zero_layernorm_backward(y, x, w, mean, rstd, dx, db=db)
    check_backward(y[-600:], x[-600:], w, mean[-600:], rstd[-600:], None, dx[-600:], None, db)
