"""Every kernel that an orthogonalisation may run, by sizes that reach it (which
they do is held on the CPU, against the rule itself): values, special matrices,
inputs far from 1, matrices behind element 2^31."""
import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests.test_gpu_muon import check_orth, gen, ns64

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32

# (count, r, c) and what runs: of gram, square and apply the tile's side, groups of
# waves, buffers (the gram product's parts), tiles that run as quarters; up to 128
# rows A and P are one kernel's work, from X or from the gram product's parts
PATHS = [
    ((3, 50, 60), "one workgroup"),
    ((2, 128, 448), "one workgroup"),
    ((200, 64, 1100), "narrow 64; 256.1.2 rest 0"),
    ((1, 64, 2000), "64.1.4 in 8, narrow 64; 64.1.4"),
    ((1, 100, 700), "narrow 128; 64.1.4"),
    ((2, 65, 449), "narrow 128; 64.1.4"),
    ((1, 128, 1024), "64.1.4 in 4, narrow 128; 64.1.4"),
    ((2, 100, 2000), "64.1.4 in 8, narrow 128; 64.1.4"),
    ((1, 200, 300), "64.1.4, 64.1.4; 64.1.4"),
    ((1, 256, 8192), "64.1.4 in 10, 64.1.4; 64.1.4"),
    ((25, 300, 500), "64.1.4, 64.1.4; 64.1.2"),
    ((40, 300, 500), "64.1.2, 64.1.2; 256.1.2 rest 0"),
    ((1, 2048, 2048), "128.2.2, 128.2.2; 128.2.2"),
    ((1, 1600, 4600), "64.1.4, 64.1.4; 128.1.2"),
    ((1, 2900, 5200), "128.1.2, 128.1.2; 256.1.2 rest 0"),
    ((1, 4096, 4400), "256.1.2 rest 0, 256.1.2 rest 0; 256.1.2 rest 32"),
    ((8, 2304, 2304), "256.1.2 rest 104, 256.1.2 rest 104; 256.1.2 rest 0"),
    ((4, 4096, 4096), "256.1.2 rest 32, 256.1.2 rest 32; 256.1.2 rest 0"),
    ((4, 2300, 2500), "256.1.2 rest 0, 256.1.2 rest 0; 256.1.2 rest 104"),
]


@pytest.mark.parametrize("size", [p[0] for p in PATHS], ids=str)
def test_each_path(size):
    count, r, c = size
    g = gen(r + c)
    u = torch.randn(count, r, c, generator=g, device="cuda") * 1e-3
    for i in range(count):  # noise, and four directions above it
        u[i] += torch.randn(r, 4, generator=g, device="cuda") @ \
            torch.randn(4, c, generator=g, device="cuda") * 3e-3
    o = torch.empty(count, r, c, dtype=BF, device="cuda")
    zs.zero_orthogonalize(u, o)
    again = torch.empty_like(o)
    zs.zero_orthogonalize(u, again)
    assert torch.equal(o, again)
    tall = torch.empty(count, c, r, dtype=BF, device="cuda")
    zs.zero_orthogonalize(u.transpose(1, 2).contiguous(), tall)
    for i in sorted({0, 1, count // 2, count - 1} & set(range(count))):
        want = ns64(u[i])
        check_orth(o[i], want, f"matrix {i}")
        check_orth(tall[i], want.t(), f"matrix {i}, tall")


# a stack on each kind of path: the one kernel, the narrow ones, the products with
# the gram product whole and in parts
STACKS = [((5, 60, 100), "one workgroup"), ((5, 100, 700), "narrow 128; 64.1.4"),
          ((5, 64, 2000), "64.1.4 in 8, narrow 64; 64.1.4"),
          ((5, 128, 1024), "64.1.4 in 4, narrow 128; 64.1.4"),
          ((5, 130, 200), "64.1.4, 64.1.4; 64.1.4"),
          ((5, 200, 9000), "64.1.4 in 7, 64.1.4; 256.1.2 rest 0"),
          ((5, 1100, 700), "64.1.4, 64.1.4; 128.1.2"),
          ((5, 1500, 1600), "128.1.2, 128.1.2; 256.1.2 rest 0")]


@pytest.mark.parametrize("size", [s[0] for s in STACKS], ids=str)
@pytest.mark.parametrize("tall", [False, True])
def test_special_matrices(size, tall):
    """Inf or NaN makes all of its matrix NaN and no other, zeros stay zero"""
    count, r, c = size
    u = torch.randn(size, generator=gen(r), device="cuda")
    u[1, r - 1, c - 1], u[2, 0, 0], u[3] = float("inf"), float("nan"), 0.0
    if tall:
        u = u.transpose(1, 2).contiguous()
    o = torch.empty(u.shape, dtype=BF, device="cuda")
    zs.zero_orthogonalize(u, o)
    assert o[1].isnan().all() and o[2].isnan().all() and (o[3] == 0).all()
    for i in (0, 4):
        check_orth(o[i], ns64(u[i]), f"matrix {i}")
    zs.zero_orthogonalize(u, o, eps=0.0)
    assert o[1:4].isnan().all() and not o[0].isnan().any() and not o[4].isnan().any()


@pytest.mark.parametrize("size", [s[0][1:] for s in STACKS], ids=str)
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_free_of_scale(size, scale):
    u = torch.randn(size, generator=gen(2), device="cuda") * scale
    for v in (u, u.t().contiguous()):
        o = torch.empty(v.shape, dtype=BF, device="cuda")
        zs.zero_orthogonalize(v, o, eps=0.0)
        check_orth(o, ns64(v, eps=0.0), str(scale))


@pytest.mark.parametrize("r,c", [(60, 100), (100, 700), (130, 200), (300, 1100)])
def test_matrices_behind_element_2_to_the_31(r, c):
    stride = (1 << 31) + 12345
    ub = torch.empty(stride + r * c, dtype=BF, device="cuda")
    ob = torch.zeros(stride + r * c, dtype=BF, device="cuda")
    u, o = (b.as_strided((2, r, c), (stride, c, 1)) for b in (ub, ob))
    u.copy_(torch.randn(2, r, c, generator=gen(r), device="cuda"))
    zs.zero_orthogonalize(u, o)
    for i in range(2):
        check_orth(o[i], ns64(u[i]), f"matrix {i}")
    assert not ob[r * c:stride].any()
