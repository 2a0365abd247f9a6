"""The Muon step's entry points on the CPU: exports, the parameter struct,
workspace sizes and refusals (all before a launch, so made-up addresses are
safe; run only where no GPU is visible)."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from zero_sharded_mixed_flatten_amd import _muon
from tests.test_lib_host import cpu_only
from tests.test_linear_host import EALIAS, EINVAL, L, ROOT, at

ERANGE = zs.ZERO_ERANGE


def test_every_declared_entry_point_is_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "zero_muon.h")).read()
    names = re.findall(r"^ZERO_API\s+[\w\s\*]*?\b(zero_\w+)\s*\(", src, flags=re.M)
    assert sorted(names) == ["zero_muon_momentum", "zero_muon_momentum_dc", "zero_muon_update",
                             "zero_muon_update_dc", "zero_orthogonalize",
                             "zero_orthogonalize_workspace_bytes"]
    for n in names:
        assert hasattr(L, n) and callable(getattr(zs, n)) and n in zs.__all__


def test_the_header_is_plain_c_and_the_struct_has_its_layout(tmp_path):
    src, exe = tmp_path / "s.c", tmp_path / "s"
    fields = [f for f, _ in _muon._NsParams._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zero_muon.h"\n'
                   "int main(void) {\n    printf(\"%zu\", sizeof(zero_ns_params));\n" +
                   "".join(f'    printf(" %zu", offsetof(zero_ns_params, {f}));\n'
                           for f in fields) +
                   '    printf(" %d", ZERO_NS_MAX_STEPS);\n    return 0;\n}\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"),
                    "-o", str(exe), str(src)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    s = _muon._NsParams
    assert out == [ctypes.sizeof(s)] + [getattr(s, f).offset for f in fields] + \
        [zs.ZERO_NS_MAX_STEPS]


def test_workspace_sizes():
    size = zs.zero_orthogonalize_workspace_bytes
    assert size(0, 5, 5) == size(1, 0, 5) == size(1, 5, 0) == 0
    assert size(1, 333, 77) == size(1, 77, 333) > 0
    # X as two pairs of planes at most, A and P, and the partial sums
    for count, r, c in ((1, 1, 1), (3, 77, 333), (48, 1600, 1600), (1, 4096, 11008)):
        rp, cp = (r + 63) // 64 * 64, (c + 63) // 64 * 64
        assert size(count, r, c) <= count * (8 * rp * cp + 4 * rp * rp + 8 * rp + 8192) + 4096
    assert size(65535, 65536, 65536) > 0
    for bad in ((-1, 1, 1), (65536, 1, 1), (1, 65537, 1), (1, 1, 65537), (1, -1, 1), (1, 1, -1)):
        with pytest.raises(ValueError):
            size(*bad)


def hp(**kw):
    return ctypes.byref(zs.AdamWHParams(**kw)._c())


def ns(steps=5, eps=1e-7, coeffs=None):
    return ctypes.byref(_muon._NsParams(steps, 0, eps, coeffs))


def control(skip=None, sumsq=None, max_norm=0.0, loss_scale=None):
    return ctypes.byref(zs._StepControl(skip, sumsq, max_norm, loss_scale))


LAY = zs.ZeroLayout(1000, 1000, 250, 1, 4, 0)
HUGE3 = (ctypes.c_double * 3)(1.0, 1e300, 1.0)
NAN3 = (ctypes.c_double * 3)(1.0, math.nan, 1.0)
MOM = dict(grads=at(1), gdt=0, rows=4, ld=300, len=250, mom=at(2), u=at(3), udt=0, nesterov=1,
           hp=hp(), ctl=None, stream=None)
MOM_DC = dict(MOM, hp=at(4))
UPD = dict(o=at(1), odt=0, master=at(2), full=at(3), wdt=0, layout=ctypes.byref(LAY), rank=1,
           off=50, len=100, hp=hp(), scale=0.2, skip=None, stream=None)
UPD_DC = dict(UPD, hp=at(4))
ORTH = dict(u=at(1), udt=0, ldu=70, su=64 * 70, count=3, rows=64, cols=70, ns=ns(), o=at(2), odt=0,
            ldo=70, so=64 * 70, ws=at(3), wsb=1 << 30, stream=None)
CALLS = {"mom": (L.zero_muon_momentum, MOM), "mom_dc": (L.zero_muon_momentum_dc, MOM_DC),
         "upd": (L.zero_muon_update, UPD), "upd_dc": (L.zero_muon_update_dc, UPD_DC),
         "orth": (L.zero_orthogonalize, ORTH)}


def status(op, **change):
    fn, base = CALLS[op]
    return fn(*{**base, **change}.values())


@cpu_only
@pytest.mark.parametrize("op,change,want", [
    ("mom", dict(gdt=3), EINVAL), ("mom", dict(udt=-1), EINVAL), ("mom", dict(rows=0), EINVAL),
    ("mom", dict(ld=249), EINVAL), ("mom", dict(len=-1), EINVAL), ("mom", dict(grads=None), EINVAL),
    ("mom", dict(mom=None), EINVAL), ("mom", dict(u=None), EINVAL), ("mom", dict(hp=None), EINVAL),
    ("mom", dict(len=(1 << 38) + 1, ld=1 << 39, rows=1), EINVAL), ("mom", dict(ld=1 << 60), EINVAL),
    ("mom", dict(grads=at(1, 1)), EINVAL), ("mom", dict(mom=at(2, 2)), EINVAL),
    ("mom", dict(udt=2, u=at(3, 2)), EINVAL), ("mom", dict(hp=hp(beta1=1.0)), EINVAL),
    ("mom", dict(hp=hp(beta1=-0.1)), EINVAL), ("mom", dict(hp=hp(grad_scale=0.0)), EINVAL),
    ("mom", dict(ctl=control(max_norm=math.nan)), EINVAL),
    ("mom", dict(u=at(2)), EALIAS), ("mom", dict(u=at(1, 600)), EALIAS),
    ("mom", dict(mom=at(1, 1804)), EALIAS), ("mom", dict(u=at(2, 996)), EALIAS),
    ("mom", dict(ctl=control(skip=at(2, 8))), EALIAS),
    ("mom", dict(ctl=control(sumsq=at(3, 8))), EALIAS),
    ("mom", dict(ctl=control(loss_scale=at(2, 8))), EALIAS),
    ("mom_dc", dict(hp=None), EINVAL), ("mom_dc", dict(hp=at(4, 4)), EINVAL),
    ("mom_dc", dict(hp=at(3, 8)), EALIAS), ("mom_dc", dict(hp=at(2, 8)), EALIAS),
    ("upd", dict(odt=2), EINVAL), ("upd", dict(wdt=2), EINVAL), ("upd", dict(layout=None), EINVAL),
    ("upd", dict(rank=4), EINVAL), ("upd", dict(rank=-1), EINVAL), ("upd", dict(off=-1), EINVAL),
    ("upd", dict(len=-1), EINVAL), ("upd", dict(off=200), ERANGE), ("upd", dict(o=None), EINVAL),
    ("upd", dict(master=None), EINVAL), ("upd", dict(full=None), EINVAL),
    ("upd", dict(o=at(1, 1)), EINVAL), ("upd", dict(master=at(2, 2)), EINVAL),
    ("upd", dict(full=at(3, 1)), EINVAL), ("upd", dict(scale=math.inf), EINVAL),
    ("upd", dict(hp=None), EINVAL), ("upd", dict(hp=hp(lr=math.nan)), EINVAL),
    ("upd", dict(hp=hp(weight_decay=-1.0)), EINVAL),
    ("upd", dict(o=at(2)), EALIAS), ("upd", dict(o=at(3, 600)), EALIAS),
    ("upd", dict(master=at(3, 700)), EALIAS), ("upd", dict(skip=at(2)), EALIAS),
    ("upd", dict(skip=at(3, 600)), EALIAS),
    ("upd_dc", dict(hp=None), EINVAL), ("upd_dc", dict(hp=at(4, 4)), EINVAL),
    ("upd_dc", dict(hp=at(2, 8)), EALIAS),
    ("orth", dict(udt=3), EINVAL), ("orth", dict(odt=2), EINVAL), ("orth", dict(count=-1), EINVAL),
    ("orth", dict(count=65536), EINVAL), ("orth", dict(rows=65537), EINVAL),
    ("orth", dict(cols=65537, ldu=1 << 20, ldo=1 << 20), EINVAL), ("orth", dict(rows=-1), EINVAL),
    ("orth", dict(ldu=69), EINVAL), ("orth", dict(ldo=69), EINVAL),
    ("orth", dict(su=64 * 70 - 1), EINVAL), ("orth", dict(so=64 * 70 - 1), EINVAL),
    ("orth", dict(su=1 << 60), EINVAL), ("orth", dict(u=None), EINVAL),
    ("orth", dict(o=None), EINVAL), ("orth", dict(u=at(1, 1)), EINVAL),
    ("orth", dict(udt=2, u=at(1, 2)), EINVAL), ("orth", dict(o=at(2, 1)), EINVAL),
    ("orth", dict(ns=ns(0)), EINVAL), ("orth", dict(ns=ns(33)), EINVAL),
    ("orth", dict(ns=ns(eps=-1.0)), EINVAL), ("orth", dict(ns=ns(eps=math.nan)), EINVAL),
    ("orth", dict(ns=ns(1, coeffs=ctypes.addressof(NAN3))), EINVAL),
    ("orth", dict(ns=ns(1, coeffs=ctypes.addressof(HUGE3))), EINVAL),
    ("orth", dict(count=65535, rows=65536, cols=65536, ldu=65536, ldo=65536, su=1 << 32,
                  so=1 << 32, wsb=1 << 62), EINVAL),
    ("orth", dict(ws=None), EINVAL), ("orth", dict(ws=at(3, 8)), EINVAL),
    ("orth", dict(wsb=1000), EINVAL), ("orth", dict(o=at(1)), EALIAS),
    ("orth", dict(o=at(1, 2 * (2 * 64 * 70))), EALIAS), ("orth", dict(ws=at(1)), EALIAS),
    ("orth", dict(ws=at(2)), EALIAS)])
def test_refusals(op, change, want):
    assert status(op, **change) == want


@cpu_only
@pytest.mark.parametrize("op,change", [
    ("mom", dict(len=0)), ("mom", dict(len=0, grads=None, mom=None, u=None)), ("upd", dict(len=0)),
    ("upd", dict(len=0, o=None, master=None, full=None)), ("orth", dict(count=0)),
    ("orth", dict(rows=0)), ("orth", dict(cols=0)), ("orth", dict(rows=0, u=None, o=None, ws=None))])
def test_empty_calls_are_no_ops(op, change):
    assert status(op, **change) == zs.ZERO_OK


def test_the_binding_refuses_what_does_not_fit():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_orthogonalize(x, x)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_muon_momentum(x, 4, 8, 8, x, x, zs.AdamWHParams())
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_muon_update(x, x, x, LAY, 0, zs.AdamWHParams())
