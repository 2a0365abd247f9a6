"""The 256 x 256 tiles of the products, their quarters after the last whole
round, and the general epilogue on both, against plain 64-bit forms; and the
weight gradient's divided 64 x 128 tiles.
tests/test_linear_plan.py holds every size here to the kernel it is meant for."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests import test_gpu_linear as small

pytestmark = pytest.mark.gpu

# (op, m, n, k, tiles, quartered): operands that are copied directly, a broken
# last step of the contraction, tiles that hang over both edges
LARGE = [("linear", 4200, 4176, 328, 289, 33),
         ("linear", 4200, 4173, 328, 289, 33),   # columns that are not whole eights
         ("linear", 4104, 2597, 584, 187, 0),
         ("dgrad", 4200, 328, 4176, 289, 33),
         ("dgrad", 4104, 584, 2600, 187, 0),
         ("wgrad", 328, 4200, 4176, 289, 33),
         ("wgrad", 584, 4104, 2600, 187, 0)]
# 64 x 128 tiles over a divided contraction
DIVIDED = ("wgrad", 4000, 40, 136)


def _of(op):
    return [c[1:4] for c in LARGE + [DIVIDED] if c[0] == op]


def _operands(rows, cols, dtype, pad, seed):
    x = small.whole(rows, cols, seed)
    ld = (cols + 7) // 8 * 8 - cols + pad        # rows 16-byte aligned
    return x, small.Box(rows, cols, dtype, 8 if pad else 0, ld, x).view


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32),
                                       (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("m,n,k", _of("linear"))
@pytest.mark.parametrize("pad", [0, 8])
def test_linear(m, n, k, pad, dtype, out):
    """whole numbers: the sum is exact and the output its one rounding"""
    print(f"\n[linear] {m} x {n} x {k} pad {pad} {dtype} -> {out}", flush=True)
    x, bx = _operands(m, k, dtype, pad, 1)
    w, bw = _operands(n, k, dtype, pad, 2)
    y = small.Box(m, n, out, 5 if pad else 0, pad)
    zs.zero_linear(bx, bw, y.view)
    torch.cuda.synchronize()
    assert torch.equal(y.view.cpu(), small.product64(x, w).to(out))
    y.untouched()


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32),
                                       (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("m,n,k", _of("dgrad"))
@pytest.mark.parametrize("pad", [0, 8])
def test_dgrad(m, n, k, pad, dtype, out):
    print(f"\n[dgrad] {m} x {n} x {k} pad {pad} {dtype} -> {out}", flush=True)
    dy, bdy = _operands(m, n, dtype, pad, 3)
    w, bw = _operands(n, k, dtype, pad, 2)
    dx = small.Box(m, k, out, 3 if pad else 0, pad)
    zs.zero_linear_dgrad(bdy, bw, dx.view)
    torch.cuda.synchronize()
    assert torch.equal(dx.view.cpu(), small.product64(dy, w.t().contiguous()).to(out))
    dx.untouched()


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.float32),
                                        (torch.float16, torch.float32),
                                        (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("m,n,k", _of("wgrad"))
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("bias", [False, True])
def test_wgrad(m, n, k, bias, pad, dtype, grad):
    """written, then accumulated: the old value widened, one rounding a time"""
    print(f"\n[wgrad] {m} x {n} x {k} bias {bias} pad {pad} {dtype} -> {grad}", flush=True)
    dy, bdy = _operands(m, n, dtype, pad, 3)
    x, bx = _operands(m, k, dtype, pad, 1)
    dw, db = small.Box(n, k, grad, 1 if pad else 0, pad), small.Box(1, n, grad, 1)
    want, sums = small.product64(dy.t().contiguous(), x.t().contiguous()), dy.sum(0)
    w, b = want.to(grad), sums.to(grad)
    for accumulate in (False, True):
        if accumulate:
            w, b = (w.double() + want).to(grad), (b.double() + sums).to(grad)
        zs.zero_linear_wgrad(bdy, bx, dw.view, db=db.view[0] if bias else None,
                             accumulate=accumulate)
        torch.cuda.synchronize()
        assert torch.equal(dw.view.cpu(), w)
        dw.untouched()
        if bias:
            assert torch.equal(db.view[0].cpu(), b)
        db.untouched()


# the general body, one row of blocks at a time: an erf GELU, ReLU, or an
# activation with a mask; and the straight ones at the same sizes
@pytest.mark.parametrize("act,p,dtype", [("gelu", 0.0, torch.bfloat16),
                                         ("relu", 0.0, torch.float16),
                                         ("gelu_tanh", 0.25, torch.bfloat16),
                                         ("silu", 0.25, torch.float16),
                                         ("gelu_tanh", 0.0, torch.bfloat16),
                                         ("none", 0.25, torch.float16)])
@pytest.mark.parametrize("m,n,k", [(4200, 4173, 328), (4104, 2597, 584)])
def test_forward_epilogues(m, n, k, act, p, dtype):
    small._forward(m, n, k, dtype, dtype, act, p, True, True)


@pytest.mark.parametrize("act,p,dtype,out", [("gelu", 0.0, torch.bfloat16, torch.bfloat16),
                                             ("relu", 0.0, torch.float16, torch.float16),
                                             ("silu", 0.25, torch.bfloat16, torch.bfloat16),
                                             ("silu", 0.0, torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("m,n,k", _of("dgrad"))
def test_dgrad_epilogues(m, n, k, act, p, dtype, out):
    small._dgrad(m, n, k, dtype, out, act, p, True)


def test_an_output_over_its_residual():
    """quarters and whole tiles, y in the place of its residual"""
    m, n, k = 4200, 4173, 328
    x, w = (small.normal(r, k, s, 0.1).to(torch.bfloat16).cuda() for r, s in ((m, 1), (n, 2)))
    r = small.normal(m, n, 3).to(torch.bfloat16).cuda()
    apart, inplace = torch.empty_like(r), r.clone()
    d = zs.ZeroDropout(0.25, seed=4)
    for act in (zs.ZERO_ACT_NONE, zs.ZERO_ACT_RELU):
        inplace.copy_(r)
        zs.zero_linear(x, w, apart, residual=r, act=act, drop=d)
        zs.zero_linear(x, w, inplace, residual=inplace, act=act, drop=d)
        assert torch.equal(apart, inplace)
