"""Which kernel a product's sizes get (CPU): the rule itself, compiled by the
host compiler, and the sizes that the GPU tests rely on, so that a changed
rule cannot move a test off the kernel it is there for."""
import ctypes
import os
import random
import subprocess

import pytest

from tests import test_gpu_linear as small
from tests.test_gpu_linear_large import DIVIDED, LARGE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OPS = {"linear": 0, "dgrad": 1, "wgrad": 2}


class Plan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("bi", "bj", "parts", "chunk", "tiles", "quartered")]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text('''#include "linear_plan.h"
using namespace zero_linear_impl;
struct Out { int64_t bi, bj, parts, chunk, tiles, quartered; };
extern "C" void plan(int op, int64_t ni, int64_t nj, int64_t nc, Out *o) {
    const Plan p = plan_for(op, ni, nj, nc);
    const int64_t tiles = ceil_div(ni, p.bi) * ceil_div(nj, p.bj);
    *o = Out{p.bi, p.bj, p.parts, p.chunk, tiles, p.bi == 256 ? quartered(tiles) : 0};
}
extern "C" int direct(uint64_t at, int64_t ld, int64_t lanes) {
    return direct_ok(reinterpret_cast<const void *>(at), ld, lanes);
}
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "zero_sharded_mixed_flatten_amd", "csrc"), str(src), "-o",
                    str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.plan.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(Plan)]
    L.direct.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64]

    def ask(op, m, n, k):
        p = Plan()
        L.plan(OPS[op], *{"linear": (m, n, k), "dgrad": (m, k, n), "wgrad": (n, k, m)}[op],
               ctypes.byref(p))
        return p

    ask.direct = lambda *a: bool(L.direct(*a))
    return ask


@pytest.mark.parametrize("op,m,n,k,tiles,quartered", LARGE)
def test_the_large_tiles_tests_reach_them(plan, op, m, n, k, tiles, quartered):
    p = plan(op, m, n, k)
    assert (p.bi, p.bj, p.parts, p.tiles, p.quartered) == (256, 256, 1, tiles, quartered)
    nc = {"linear": k, "dgrad": n, "wgrad": m}[op]
    assert nc % 64 != 0 and nc > 64
    # rows of whole pieces, so that the direct path runs
    lanes = {"linear": (0, 0), "dgrad": (0, k), "wgrad": (n, k)}[op]
    assert all(plan.direct(1 << 20, 4208, at) for at in lanes)


def test_the_small_tests_reach_the_other_kernels(plan):
    """few rows, both small tiles, whole and divided, over the lists of sizes"""
    kinds = {op: set() for op in OPS}
    for m, n, k in small.SIZES:
        for op in OPS:
            p = plan(op, m, n, k)
            kinds[op].add((p.bi, p.parts > 1))
    tiles = {(64, False), (64, True), (128, False), (128, True)}
    assert kinds["linear"] >= tiles | {(16, False), (32, False)}
    assert kinds["dgrad"] >= tiles and kinds["wgrad"] >= tiles - {(64, True)}
    p = plan(*DIVIDED)
    assert DIVIDED[0] == "wgrad" and p.bi == 64 and p.parts > 1
    for m, n, k in small.STRAIGHT:
        p = plan("linear", m, n, k)
        assert p.parts == 1 and p.bi == (256 if m > 1000 else 128)


def test_what_is_copied_directly(plan):
    assert plan.direct(16, 8, 8) and plan.direct(16, 8, 0)
    assert not plan.direct(8, 8, 8)            # a start off 16 bytes
    assert not plan.direct(16, 9, 0)           # rows off 16 bytes
    assert not plan.direct(16, 8, 12)          # rows that end inside a piece
    assert not plan.direct(16, 1 << 22, 0)     # a tile's rows past 32 bits


def test_parts_cover_the_contraction_once(plan):
    rng = random.Random(1)
    for _ in range(3000):
        op = rng.choice(list(OPS))
        m, n, k = (int(2 ** rng.uniform(0, 16)) for _ in range(3))
        p, nc = plan(op, m, n, k), {"linear": k, "dgrad": n, "wgrad": m}[op]
        assert p.parts >= 1 and p.tiles >= 1 and 0 <= p.quartered <= 128
        if p.bi > 32:
            assert p.chunk % 64 == 0 and p.parts * p.chunk >= nc > (p.parts - 1) * p.chunk
        if p.parts > 1:                         # all of them on the card at once
            assert p.bi <= 128 and p.tiles * p.parts <= 512
        if p.bi <= 32:
            assert op == "linear" and m <= 32 and p.parts == 1


def test_few_rows(plan):
    """the few-rows kernel up to 16 rows; from 17 on only where no CU has more
    than 6400 of the contraction to do"""
    for m, n, k in [(1, 48, 12288), (16, 50257, 1600), (16, 4096, 11008), (17, 1600, 1600),
                    (32, 4096, 4096), (32, 4096, 6400), (32, 6400, 2048), (32, 2000, 200)]:
        p = plan("linear", m, n, k)
        assert (p.bi, p.parts) == (16 if m <= 16 else 32, 1)
    for m, n, k in [(32, 48, 12288), (17, 1024, 12288), (32, 4096, 11008), (32, 11008, 4096),
                    (24, 32000, 2048), (32, 6400, 6400)]:
        p = plan("linear", m, n, k)
        assert p.bi == 64
