"""zero_dropout against the mask's definition in NumPy: every output bit."""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
CANARY = 55.0


def _want(x, r, p, seed, stream, row0=0):
    """scale and select in fp32, residual added in fp32, one rounding"""
    v = torch.where(ref.keep(*x.shape, p, seed, stream, row0),
                    x.float() * np.float32(ref.scale32(p)), torch.zeros(()))
    return (v if r is None else r.float() + v).to(x.dtype)


def _rows(rows, cols, dtype, pad, lead, seed):
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(lead + rows * (cols + pad), generator=g).to(dtype).cuda()
    return buf[lead:].view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols,pad,lead", [(1, 1, 0, 0), (1, 1600, 0, 0), (3, 15, 2, 1),
                                                (5, 31, 1, 0), (7, 32, 0, 0), (4, 33, 3, 2),
                                                (2, 48, 0, 4), (257, 100, 4, 0), (1000, 333, 0, 0),
                                                (64, 4096, 8, 8)])
@pytest.mark.parametrize("p,res", [(0.1, False), (0.5, True)])
def test_every_bit(rows, cols, pad, lead, dtype, p, res):
    print(f"\n[dropout] {rows} x {cols} pad {pad} lead {lead} {dtype} p {p} res {res}", flush=True)
    seed, offset, row0 = 0xFEDCBA9876543210, 0x1FFFFFFFF, 123456
    x = _rows(rows, cols, dtype, pad, lead, 1)
    r = _rows(rows, cols, dtype, pad, lead, 2) if res else None
    buf = torch.full((lead + rows * (cols + pad) + 40,), CANARY, dtype=dtype, device="cuda")
    y = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    zs.zero_dropout(x, y, zs.ZeroDropout(p, seed, offset, row0), residual=r)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), _want(x.cpu(), None if r is None else r.cpu(), p, seed, offset, row0))
    y.fill_(CANARY)
    assert bool((buf == CANARY).all())


@pytest.mark.parametrize("p", [0.0, 1e-9, 1.0 / 65536, 0.25, 0.9999999])
def test_the_probability_s_ends(p):
    """p of no drop is the identity bit for bit; the threshold stops at 65535"""
    x = _rows(64, 500, torch.float32, 0, 0, 3)
    y = torch.empty_like(x)
    zs.zero_dropout(x, y, zs.ZeroDropout(p, 9))
    assert torch.equal(y.cpu(), _want(x.cpu(), None, p, 9, 0))
    if ref.threshold(p) == 0:
        assert torch.equal(x, y)


def test_in_place_backward_and_split_rows():
    x = _rows(100, 70, torch.bfloat16, 0, 0, 4)
    d = zs.ZeroDropout(0.3, 77, 5)
    y = torch.empty_like(x)
    zs.zero_dropout(x, y, d)
    kept = y != 0
    # the backward pass draws the same mask
    dy, dx = torch.ones_like(x), torch.empty_like(x)
    zs.zero_dropout(dy, dx, d)
    assert torch.equal(dx != 0, ref.keep(100, 70, 0.3, 77, 5).cuda())
    assert bool((kept <= (dx != 0)).all())
    # in the place of x, of the residual, and in two calls of rows
    z = x.clone()
    zs.zero_dropout(z, z, d)
    assert torch.equal(z, y)
    r = _rows(100, 70, torch.bfloat16, 0, 0, 5)
    a, b = torch.empty_like(r), r.clone()
    zs.zero_dropout(x, a, d, residual=r)
    zs.zero_dropout(x, b, d, residual=b)
    assert torch.equal(a, b)
    halves = torch.empty_like(x)
    zs.zero_dropout(x[:37], halves[:37], d)
    zs.zero_dropout(x[37:], halves[37:], zs.ZeroDropout(0.3, 77, 5, row0=37))
    assert torch.equal(halves, y)


def test_dropped_values_are_zero_whatever_they_were():
    x = torch.full((50, 64), math.nan, device="cuda")
    x[::2] = math.inf
    y = torch.empty_like(x)
    zs.zero_dropout(x, y, zs.ZeroDropout(0.5, 1))
    keep = ref.keep(50, 64, 0.5, 1, 0)
    assert bool((y.cpu()[~keep] == 0).all()) and not bool(torch.isfinite(y.cpu()[keep]).any())


def test_kept_share():
    """2^22 elements at p = 0.3: the kept count is within 5 standard
    deviations of its mean, in every column class of the mask too"""
    x = torch.ones(4096, 1024, device="cuda")
    y = torch.empty_like(x)
    zs.zero_dropout(x, y, zs.ZeroDropout(0.3, 2024, 7))
    q = 1 - ref.threshold(0.3) / 65536
    for cols in [slice(None)] + [slice(c, None, 32) for c in range(32)]:
        part = y[:, cols]
        n = part.numel()
        assert abs(float((part != 0).sum()) - n * q) < 5 * math.sqrt(n * q * (1 - q))


def test_a_captured_graph_draws_a_new_mask_every_replay():
    """the step counter in device memory moves the stream; every replay
    equals the eager call of that step"""
    x = _rows(40, 96, torch.bfloat16, 0, 0, 6)
    w = _rows(64, 96, torch.bfloat16, 0, 0, 7)
    t = zs.new_step_counter(1)
    y, h = torch.empty_like(x), torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    d = zs.ZeroDropout(0.4, 31, 1000, step=t)
    ws = torch.empty(max(1, zs.zero_linear_workspace_bytes(zs.ZERO_LINEAR, 40, 64, 96)),
                     dtype=torch.uint8, device="cuda")

    def work():
        zs.zero_dropout(x, y, d)
        zs.zero_linear(x, w, h, drop=d, workspace=ws)
        zs.zero_step_counter_advance(t)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    t.fill_(1)
    for step in range(1, 6):
        graph.replay()
        torch.cuda.synchronize()
        assert int(t.item()) == step + 1
        eager, eh = torch.empty_like(y), torch.empty_like(h)
        zs.zero_dropout(x, eager, zs.ZeroDropout(0.4, 31, 1000 + step))
        zs.zero_linear(x, w, eh, drop=zs.ZeroDropout(0.4, 31, 1000 + step))
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(h, eh)
        assert torch.equal(y.cpu(), _want(x.cpu(), None, 0.4, 31, 1000 + step))


def test_more_than_one_launch():
    """2^33 elements and more go out as several launches; the last rows and
    those about the first launch's end against the definition"""
    rows, cols = (1 << 21) + 37, 4096
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    zs.zero_dropout(x, x, zs.ZeroDropout(0.5, 8))
    torch.cuda.synchronize()
    for first in (0, (1 << 21) - 8, rows - 16):
        keep = ref.keep(16, cols, 0.5, 8, 0, first)
        assert torch.equal(x[first:first + 16].cpu() != 0, keep)
    del x
    torch.cuda.empty_cache()
