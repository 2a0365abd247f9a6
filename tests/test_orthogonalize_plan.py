"""Which kernels an orthogonalisation's sizes get, and each round's constants
(CPU): the rules themselves, compiled by the host compiler, and the sizes that
the GPU tests rely on, so that a changed rule cannot move a test off the kernel
it is there for."""
import ctypes
import os
import random
import subprocess

import pytest

import zero_sharded_mixed_flatten_amd as zs
from tests.test_gpu_orthogonalize_paths import PATHS, STACKS
from zero_sharded_mixed_flatten_amd import _muon

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GRAM, SQUARE, APPLY = range(3)


class Way(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in
                ("small", "rp", "side", "groups", "buffers", "parts", "steps", "all", "rest",
                 "bytes")]


class Round(ctypes.Structure):
    _fields_ = [(f, ctypes.c_float) for f in
                ("a", "b", "c", "lo_share", "lo_rest", "to_a", "from_a", "from_aa", "to_p",
                 "from_p")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = d / "plan.cpp", d / "plan.so"
    src.write_text('''#include "orthogonalize_plan.h"
using namespace zero_muon_impl;
struct Out { int64_t small, rp, side, groups, buffers, parts, steps, all, rest, bytes; };
extern "C" void way(int kind, int64_t count, int64_t rows, int64_t cols, Out *o) {
    const Work w = work_of(count, rows, cols);
    const Way p = way_of(kind, w, count);
    *o = Out{is_small(w), w.rp, p.side, p.groups, p.buffers, p.parts, p.steps,
             (kind == GRAM ? w.cp : w.rp) / kBK, rest_of(kind, w, count), w.bytes};
}
extern "C" void rounds(const zero_ns_params *k, int64_t r, Round *o) { rounds_of(*k, r, o); }
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "zero_sharded_mixed_flatten_amd", "csrc"), str(src), "-o",
                    str(out)], check=True)
    L = ctypes.CDLL(str(out))
    L.way.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(Way)]
    L.rounds.argtypes = [ctypes.POINTER(_muon._NsParams), ctypes.c_int64, ctypes.POINTER(Round)]
    return L


def way(lib, kind, size):
    w = Way()
    lib.way(kind, *size, ctypes.byref(w))
    return w


def path(lib, size):
    g, s, a = (way(lib, k, size) for k in (GRAM, SQUARE, APPLY))
    if g.small:
        return "one workgroup"

    def name(w):
        return f"{w.side}.{w.groups}.{w.buffers}" + (f" in {w.parts}" if w.parts > 1 else "") + \
            (f" rest {w.rest}" if w.side == 256 else "")

    if g.rp > 128:
        return f"{name(g)}, {name(s)}; {name(a)}"
    return (name(g) + ", " if g.parts > 1 else "") + f"narrow {g.rp}; {name(a)}"


@pytest.mark.parametrize("size,want", PATHS + STACKS, ids=str)
def test_the_gpu_tests_reach_their_kernels(lib, size, want):
    assert path(lib, size) == want
    count, r, c = size
    assert path(lib, (count, c, r)) == want


def test_every_kernel_is_among_them(lib):
    """what a call of any size may launch, a GPU test launches"""
    def launches(size):
        ways = [way(lib, k, size) for k in (GRAM, SQUARE, APPLY)]
        if ways[0].small:
            return {("one", ways[0].rp)}
        out = set()
        narrow = ways[0].rp <= 128
        if narrow:
            out.add(("narrow", ways[0].rp, ways[0].parts > 1))
        for k, w in enumerate(ways):
            if narrow and (k == SQUARE or (k == GRAM and w.parts == 1)):
                continue
            out.add((k, w.side, w.groups, w.buffers))
            if k == GRAM and w.parts > 1 and not narrow:
                out.add("join")
            if w.rest:
                out.add((k, "quarters", 1 if w.rest > 64 else 2))
        return out

    tested = set().union(*(launches(p[0]) for p in PATHS + STACKS))
    rng = random.Random(1)
    met = set()
    for _ in range(20000):
        size = (int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 14)),
                int(2 ** rng.uniform(0, 16)))
        met |= launches(size)
    assert met <= tested, met - tested


def test_parts_cover_the_contraction_once(lib):
    rng = random.Random(2)
    for _ in range(5000):
        size = (int(2 ** rng.uniform(0, 8)), int(2 ** rng.uniform(0, 14)),
                int(2 ** rng.uniform(0, 16)))
        for kind in (GRAM, SQUARE, APPLY):
            w = way(lib, kind, size)
            assert (w.parts - 1) * w.steps < w.all <= w.parts * w.steps
            assert w.bytes == zs.zero_orthogonalize_workspace_bytes(*size)


# ---------------------------------------------------------------------------
# a round's constants


def rounds(lib, coeffs, r=64):
    flat = None
    if coeffs is not None:
        flat = (ctypes.c_double * (3 * len(coeffs)))(*[v for abc in coeffs for v in abc])
    n = 5 if coeffs is None else len(coeffs)
    out = (Round * n)()
    ns = _muon._NsParams(n, 0, 1e-7, None if flat is None else ctypes.addressof(flat))
    lib.rounds(ctypes.byref(ns), r, out)
    return out


def test_the_usual_rounds(lib):
    for q in rounds(lib, None):
        assert (q.a, q.b, q.c) == tuple(ctypes.c_float(v).value for v in (3.4445, -4.7750, 2.0315))
        assert (q.to_a, q.from_a, q.from_aa, q.to_p, q.from_p) == \
            (2.0 ** -12, 2.0 ** -12, 2.0 ** -24, 2.0 ** 12, 2.0 ** -12)
    assert [q.lo_share for q in rounds(lib, None)] == [0, 0, 0, 1, 1]
    assert [q.lo_rest != 0 for q in rounds(lib, None)] == [True, True, True, False, False]
    assert [q.lo_share for q in rounds(lib, None, r=1)] == [1] * 5


def test_off_diagonals_fit_fp16_for_any_singular_values_allowed(lib):
    """against the polynomial on a grid of singular values, round by round"""
    rng = random.Random(3)
    for _ in range(400):
        coeffs = [tuple(rng.choice([0.0, rng.uniform(-4, 4), 10 ** rng.uniform(-3, 3)])
                        for _ in range(3)) for _ in range(rng.randint(1, 6))]
        top = 1.0
        for (a, b, c), q in zip(coeffs, rounds(lib, coeffs)):
            s = [top * k / 2000 for k in range(2001)]
            off_a = top * top / 2
            p = [b * x ** 2 + c * x ** 4 for x in s]
            off_p = (max(p) - min(p)) / 2
            # the scale of A in fp16 is to_a x 2^24 a unit
            assert off_a * q.to_a * 2.0 ** 24 <= 65504 and off_p * q.to_p <= 65504
            assert q.to_a * 2.0 ** 24 * q.from_a == 1 and q.to_p * q.from_p == 1
            assert q.from_aa == q.from_a ** 2
            # and no smaller than it has to be
            assert q.to_a == 2.0 ** -12 or off_a * q.to_a * 2.0 ** 24 > 8000 or top >= 15
            top = min(15.9, max(abs(x * (a + y)) for x, y in zip(s, p)))
