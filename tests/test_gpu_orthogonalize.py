"""The orthogonalisation where its roundings are hardest on it: matrices of a
few strong directions, carried by all rows or by few of them, against the
definition in 64 bits.

Tolerance.  A round's fp16 operands (O, Q and X's high half) are off by u =
2^-11 of an element at most, by 2^-12.3 in the root mean square, and X's low
half is as large as that rounding.  Where many elements add up the mean counts:
two operands a product and |b s^2 + c s^4| <= 2.81 bring a round to below 4 x
2^-12.3 of the result's norm, and five rounds, added in squares with the
polynomial's slope at their values (below 2 in the square mean), to below
2^-9.  That holds if no round's error reaches the small directions, which
every later round multiplies by 3.4445: with an error of 2^-12 there after the
first round, 141 times that is 3e-2 at the end.  Where fewer than 16 rows or
columns carry the matrix a product adds up too few elements for the mean, and
the largest rounding counts: u / 2^-12.3 = 2.5 times as much.  The result adds
half a step of its type."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests.test_gpu_muon import gen, ns64

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def error(o, u, **kw):
    want = ns64(u, **kw)
    return ((o.double() - want).norm() / want.norm()).item()


def allowed(t, carriers, rounds=1.0):
    return 2.0 ** -9 * rounds * (1.0 if carriers >= 16 else 2.5) + torch.finfo(t).eps / 2


def check(u, carriers, what, rounds=1.0, **kw):
    for v in (u, u.t().contiguous()):
        o = torch.empty(v.shape, dtype=HF, device="cuda")
        zs.zero_orthogonalize(v, o, **kw)
        err, tol = error(o, v, **kw), allowed(HF, carriers, rounds)
        assert err <= tol, f"{tuple(v.shape)} {what}: {err:.3g} off, {tol:.3g} allowed"


# one workgroup a matrix; up to 128 rows and longer; the products' tiles
SHAPES = [(8, 8), (16, 256), (64, 64), (64, 512), (64, 1024), (128, 448), (65, 300), (50, 1500),
          (100, 700), (128, 2000), (130, 200), (200, 200), (300, 520), (512, 512), (700, 1100)]


@pytest.mark.parametrize("r,c", SHAPES)
@pytest.mark.parametrize("directions", [1, 2, 8])
def test_strong_directions_over_noise(r, c, directions):
    for noise in (1e-3, 1e-6):
        g = gen(r + c + directions)
        u = torch.randn(r, directions, generator=g, device="cuda") @ \
            torch.randn(directions, c, generator=g, device="cuda")
        u = (u + noise * torch.randn(r, c, generator=g, device="cuda")).to(BF)
        check(u, min(r, c), f"{directions} directions over {noise}")


@pytest.mark.parametrize("r,c", [(64, 64), (40, 900), (128, 448), (90, 1500), (130, 200),
                                 (300, 520), (1024, 1024), (700, 2300)])
@pytest.mark.parametrize("rows", [2, 4, 16])
def test_one_direction_carried_by_few_rows(r, c, rows):
    """as a layer whose other units are all but dead"""
    for both in (False, True):
        g = gen(r + c + rows + both)
        a = torch.zeros(r, 1, device="cuda")
        b = torch.randn(1, c, generator=g, device="cuda")
        a[:rows] = torch.randn(rows, 1, generator=g, device="cuda")
        if both:
            b[:, rows:] = 0
        u = (a @ b + 1e-6 * torch.randn(r, c, generator=g, device="cuda")).to(BF)
        check(u, rows, f"{rows} rows, few columns: {both}")


@pytest.mark.parametrize("r,c", [(1, 1), (1, 8), (1, 300), (3, 9), (16, 16), (64, 1024), (128, 448),
                                 (128, 1024), (512, 2048)])
def test_full_rank(r, c):
    for seed in range(3):
        u = torch.randn(r, c, generator=gen(seed), device="cuda").to(BF)
        check(u, min(r, c), "full rank")
    if r > 1:
        check(torch.linalg.qr(torch.randn(c, r, generator=gen(9), device="cuda"))[0].t()
              .contiguous(), min(r, c), "orthogonal rows")


def test_rounds_whose_slope_is_not_the_usual():
    """which rounds keep small directions free of X's low half goes by the
    coefficients; |b s^2 + c s^4| is 8.1 in the first of the steep ones, 2.9 times
    the usual, which makes the sum of squares of five rounds (4 + 2.9^2) / 5 = 1.6^2
    times as large"""
    steep = [(8.2, -23.0, 16.5), (4.0, -2.9, 0.55), (3.8, -2.8, 0.53), (3.3, -2.4, 0.46),
             (2.3, -1.6, 0.4)]
    flat = [(1.5, -0.5, 0.0)] * 8
    for coeffs in (steep, flat):
        for r, c in ((16, 256), (64, 700), (200, 300)):
            g = gen(r)
            u = (torch.randn(r, 1, generator=g, device="cuda") @
                 torch.randn(1, c, generator=g, device="cuda") +
                 1e-4 * torch.randn(r, c, generator=g, device="cuda")).to(BF)
            check(u, r, str(coeffs[0]), 1.6, steps=len(coeffs), coeffs=coeffs)


LARGE = [([(1.5, 0.0, 0.0)] * 6, 1.0),                      # singular value 11.4
         ([(6.0, 0.0, 0.0), (0.2, 0.0, 0.0)], 1.0),
         ([(15.5, 0.0, 0.0), (0.05, 0.0, 0.0)], 1.0),
         ([(12.0, 0.0, 0.0), (0.5, -0.004, 1e-5)], 1.0),
         ([(61.0, -60.0, 0.0), (1.0, 0.0, 0.0)], 60 / 2.81)]  # an off-diagonal of P is -30


@pytest.mark.parametrize("coeffs,rounds", LARGE)
@pytest.mark.parametrize("r,c", [(1, 1), (2, 2), (64, 64), (30, 1000), (128, 448), (100, 700),
                                 (128, 2000), (40, 1500), (200, 300), (300, 520), (1024, 1024)])
def test_singular_values_up_to_the_documented_limit(r, c, coeffs, rounds):
    """all of the matrix in two rows: the off-diagonals of A are half the square of
    the singular value.  An error is multiplied by |b s^2 + c s^4| as far as that
    is larger than the usual."""
    u = torch.zeros(r, c, device="cuda")
    u[:2] = torch.rand(1, c, generator=gen(c), device="cuda") + 0.5
    check(u.to(BF), 2, str(coeffs), rounds, steps=len(coeffs), coeffs=coeffs)
