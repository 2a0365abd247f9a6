"""The layer products and the dropout on the CPU: exports, workspace sizes
and refusals (everything here is refused before a launch, so made-up
addresses are safe; run only where no GPU is visible)."""
import ctypes
import math
import os
import re

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from zero_sharded_mixed_flatten_amd import _linear
from tests.test_lib_host import cpu_only

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = zs._lib
EINVAL, EALIAS = zs.ZERO_EINVAL, zs.ZERO_EALIAS
BIG = (1 << 31) - 1024


def at(i, off=0):
    return (1 << 40) + i * (1 << 36) + off


def test_every_declared_entry_point_is_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "zero_linear.h")).read()
    names = re.findall(r"^ZERO_API\s+[\w\s\*]*?\b(zero_\w+)\s*\(", src, flags=re.M)
    assert sorted(names) == ["zero_dropout", "zero_linear", "zero_linear_dgrad",
                             "zero_linear_wgrad", "zero_linear_workspace_bytes"]
    for n in names:
        assert hasattr(L, n) and callable(getattr(zs, n)) and n in zs.__all__


def test_the_header_is_plain_c_and_the_struct_has_its_layout(tmp_path):
    import subprocess
    src, exe = tmp_path / "s.c", tmp_path / "s"
    fields = [f for f, _ in _linear._DropoutParams._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zero_linear.h"\n'
                   "int main(void) {\n    printf(\"%zu\", sizeof(zero_dropout_params));\n" +
                   "".join(f'    printf(" %zu", offsetof(zero_dropout_params, {f}));\n'
                           for f in fields) +
                   '    printf(" %d %d %d", ZERO_ACT_SILU, ZERO_LINEAR, ZERO_LINEAR_WGRAD);\n'
                   "    return 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"),
                    "-o", str(exe), str(src)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    s = _linear._DropoutParams
    assert out == [ctypes.sizeof(s)] + [getattr(s, f).offset for f in fields] + \
        [zs.ZERO_ACT_SILU, zs.ZERO_LINEAR, zs.ZERO_LINEAR_WGRAD]


def test_workspace_sizes():
    for op in (zs.ZERO_LINEAR, zs.ZERO_LINEAR_DGRAD, zs.ZERO_LINEAR_WGRAD):
        assert zs.zero_linear_workspace_bytes(op, 0, 5, 7) >= 0
        assert zs.zero_linear_workspace_bytes(op, 8192, 4096, 11008) == 0
        for bad in ((-1, 1, 1), (1, BIG + 1, 1), (1, 1, -1)):
            with pytest.raises(ValueError):
                zs.zero_linear_workspace_bytes(op, *bad)
        # the parts of a divided contraction stay a bounded scratch
        for m, n, k in ((1, 6400, 1600), (16, 4096, 11008), (333, 333, 1 << 20), (1, 1, BIG)):
            assert zs.zero_linear_workspace_bytes(op, m, n, k) < 1 << 34
    for op in (-1, 3):
        with pytest.raises(ValueError):
            zs.zero_linear_workspace_bytes(op, 1, 1, 1)


def drop(p=0.1, row0=0, step=None):
    return ctypes.byref(_linear._DropoutParams(p, 1, 2, row0, step))


FWD = dict(x=at(1), dt=0, ldx=64, w=at(2), ldw=64, bias=at(3), m=32, n=48, k=64, act=0, drop=None,
           res=at(4), ldr=48, y=at(5), ydt=0, ldy=48, z=at(6), ldz=48, ws=at(7), wsb=1 << 30,
           stream=None)
DGRAD = dict(dy=at(1), dt=0, lddy=48, w=at(2), ldw=64, m=32, n=48, k=64, act=4, z=at(3), ldz=64,
             drop=None, res=at(4), ldr=64, dx=at(5), dxdt=0, lddx=64, ws=at(6), wsb=1 << 30,
             stream=None)
WGRAD = dict(dy=at(1), dt=0, lddy=48, x=at(2), ldx=64, m=32, n=48, k=64, dw=at(3), gdt=2, lddw=64,
             db=at(4), acc=0, ws=at(5), wsb=1 << 30, stream=None)
DROP = dict(x=at(1), dt=0, ldx=64, rows=32, cols=64, drop=drop(), res=at(2), ldr=64, y=at(3),
            ldy=64, stream=None)
CALLS = {"linear": (L.zero_linear, FWD), "dgrad": (L.zero_linear_dgrad, DGRAD),
         "wgrad": (L.zero_linear_wgrad, WGRAD), "dropout": (L.zero_dropout, DROP)}


def status(op, **change):
    fn, base = CALLS[op]
    return fn(*{**base, **change}.values())


LONG = dict(m=40, n=8, k=1 << 16)   # a divided contraction for linear


@cpu_only
@pytest.mark.parametrize("op,change,want", [
    ("linear", dict(dt=2), EINVAL), ("linear", dict(dt=9), EINVAL), ("linear", dict(ydt=1), EINVAL),
    ("linear", dict(act=5), EINVAL), ("linear", dict(act=-1), EINVAL),
    ("linear", dict(m=-1), EINVAL), ("linear", dict(n=BIG + 1, ldy=1 << 33, ldr=1 << 33, ldz=1 << 33), EINVAL),
    ("linear", dict(ldx=63), EINVAL), ("linear", dict(ldw=63), EINVAL),
    ("linear", dict(ldy=47), EINVAL), ("linear", dict(ldr=47), EINVAL),
    ("linear", dict(ldz=47), EINVAL), ("linear", dict(x=None), EINVAL),
    ("linear", dict(w=None), EINVAL), ("linear", dict(y=None), EINVAL),
    ("linear", dict(x=at(1, 1)), EINVAL), ("linear", dict(ydt=2, y=at(5, 2)), EINVAL),
    ("linear", dict(ldx=1 << 60), EINVAL),
    ("linear", dict(drop=drop(1.0)), EINVAL), ("linear", dict(drop=drop(-0.1)), EINVAL),
    ("linear", dict(drop=drop(math.nan)), EINVAL), ("linear", dict(drop=drop(row0=-1)), EINVAL),
    ("linear", dict(drop=drop(row0=(1 << 32) - 31)), EINVAL),
    ("linear", dict(drop=drop(step=at(9, 4))), EINVAL),
    ("linear", dict(drop=drop(step=at(5, 8))), EALIAS),
    ("linear", dict(y=at(1, 64)), EALIAS), ("linear", dict(y=at(2)), EALIAS),
    ("linear", dict(y=at(3)), EALIAS), ("linear", dict(y=at(6)), EALIAS),
    ("linear", dict(z=at(1)), EALIAS), ("linear", dict(z=at(4)), EALIAS),
    ("linear", dict(res=at(5, 2)), EALIAS), ("linear", dict(res=at(5), ldr=50), EALIAS),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=None), EINVAL),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=at(7, 8)), EINVAL),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, wsb=16), EINVAL),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=at(1)), EALIAS),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=at(5)), EALIAS),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=at(4)), EALIAS),
    ("linear", dict(LONG, ldx=1 << 16, ldw=1 << 16, ws=at(6)), EALIAS),
    # more output tiles than one launch takes
    ("dgrad", dict(m=1, n=1, k=BIG, ldw=BIG, lddx=BIG, act=0, res=None), EINVAL),
    ("dgrad", dict(dt=2), EINVAL), ("dgrad", dict(dxdt=1), EINVAL), ("dgrad", dict(z=None), EINVAL),
    ("dgrad", dict(lddy=47), EINVAL), ("dgrad", dict(lddx=63), EINVAL),
    ("dgrad", dict(ldz=63), EINVAL), ("dgrad", dict(act=7), EINVAL),
    ("dgrad", dict(dx=at(1)), EALIAS), ("dgrad", dict(dx=at(2)), EALIAS),
    ("dgrad", dict(dx=at(3)), EALIAS), ("dgrad", dict(res=at(5, 4)), EALIAS),
    ("wgrad", dict(dt=2), EINVAL), ("wgrad", dict(gdt=1), EINVAL), ("wgrad", dict(dw=None), EINVAL),
    ("wgrad", dict(lddw=63), EINVAL), ("wgrad", dict(ldx=60), EINVAL),
    ("wgrad", dict(dw=at(3, 2)), EINVAL), ("wgrad", dict(db=at(4, 1)), EINVAL),
    ("wgrad", dict(k=0), EINVAL),
    ("wgrad", dict(dw=at(1)), EALIAS), ("wgrad", dict(db=at(2)), EALIAS),
    ("wgrad", dict(db=at(3, 16)), EALIAS),
    ("wgrad", dict(m=1 << 16, ws=None), EINVAL), ("wgrad", dict(m=1 << 16, wsb=64), EINVAL),
    ("wgrad", dict(m=1 << 16, ws=at(3)), EALIAS), ("wgrad", dict(m=1 << 16, ws=at(4)), EALIAS),
    ("dropout", dict(drop=None), EINVAL), ("dropout", dict(dt=3), EINVAL),
    ("dropout", dict(rows=-1), EINVAL), ("dropout", dict(ldx=63), EINVAL),
    ("dropout", dict(drop=drop(1.5)), EINVAL), ("dropout", dict(x=None), EINVAL),
    ("dropout", dict(y=at(1, 2)), EALIAS), ("dropout", dict(y=at(1), ldy=65), EALIAS),
    ("dropout", dict(y=at(2), ldy=80), EALIAS), ("dropout", dict(drop=drop(step=at(3))), EALIAS),
])
def test_refusals(op, change, want):
    assert status(op, **change) == want


@cpu_only
@pytest.mark.parametrize("op,change", [
    ("linear", dict(m=0)), ("linear", dict(n=0)), ("linear", dict(m=0, x=None, y=None, z=None, res=None)),
    ("dgrad", dict(m=0)), ("dgrad", dict(k=0)), ("wgrad", dict(n=0)), ("wgrad", dict(k=0, db=None)),
    ("dropout", dict(rows=0)), ("dropout", dict(cols=0))])
def test_empty_outputs_are_no_ops(op, change):
    assert status(op, **change) == zs.ZERO_OK


def test_the_binding_refuses_what_is_not_a_gpu_matrix():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_linear(x, x, x)
    with pytest.raises(TypeError, match="16-bit"):
        zs.zero_linear(x.float(), x, x)
    with pytest.raises(TypeError, match="16-bit"):
        zs.zero_linear_wgrad(x.float(), x, x)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_dropout(x, x, zs.ZeroDropout(0.1))
