"""The layer norm at the edges of its domain.  Finite rows whose squares pass
fp32's range: 1 / sqrt of an infinite variance is 0, so y is the bias (or 0), as
fp32 arithmetic has it.  Calls whose 16-bit type only the gradients tell."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


# a fraction of a wave a row, one wave, several, a loop
@pytest.mark.parametrize("n", [2, 7, 8, 100, 200, 500, 1600, 4096, 9001, 16384, 20000])
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("m", [3, 700])
def test_squares_beyond_the_range(n, xt, m):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x = torch.randn(m, n, generator=g, device="cuda")
    x[1, ::2], x[1, 1::2] = 1e30, 3e30     # a mean: its square passes the range too
    x[2, ::2], x[2, 1::2] = -2e25, 2e25
    x = x.to(xt)
    w, b = (torch.randn(n, generator=g, device="cuda").to(BF) for _ in range(2))
    y = torch.empty(m, n, device="cuda")
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    zs.zero_layernorm(x, w, b, y, mean=mean, rstd=rstd)
    assert (rstd[1:3] == 0).all()
    assert torch.equal(y[1:3], b.float().expand(2, n))
    want = x[1].double().mean()
    assert (mean[1].double() - want).abs() <= 2.0 ** -16 * want
    others = [0] + list(range(3, m))
    assert torch.isfinite(y[others]).all() and (rstd[others] > 0).all()
    dy, dx = torch.ones_like(y), torch.empty_like(x)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx)
    assert (dx[1:3] == 0).all()


@pytest.mark.parametrize("n", [8, 100, 1600, 20000])
def test_a_sum_beyond_the_range_is_nan(n):
    x = torch.ones(3, n, device="cuda", dtype=BF)
    x[1] = 3e38
    y, rstd = torch.empty(3, n, device="cuda"), torch.empty(3, device="cuda")
    zs.zero_layernorm(x, None, None, y, rstd=rstd)
    assert y[1].isnan().all() and (y[[0, 2]] == 0).all()


@pytest.mark.parametrize("gt", [BF, torch.float16])
def test_gradients_in_16_bits_of_fp32_rows_without_a_weight(gt):
    """the gradient row's type is then the only 16-bit one of the call"""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    m, n = 40, 300
    x, dy = (torch.randn(m, n, generator=g, device="cuda") for _ in range(2))
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    zs.zero_layernorm(x, None, None, torch.empty_like(x), mean=mean, rstd=rstd)
    dx, grads = torch.empty_like(x), []
    for t in (gt, F):
        dw, db = (torch.empty(n, dtype=t, device="cuda") for _ in range(2))
        zs.zero_layernorm_backward(dy, x, None, mean, rstd, dx, dw=dw, db=db)
        zs.zero_layernorm_backward(dy, x, None, mean, rstd, dx, db=torch.empty_like(db))
        grads.append((dw, db))
    for a, b in zip(*grads):
        assert torch.equal(a, b.to(gt))  # one sum, rounded once
