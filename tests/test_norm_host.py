"""The layer norm on the CPU: exports, workspace sizes and refusals
(everything here is refused before a launch, so made-up addresses are safe;
run only where no GPU is visible)."""
import math
import os
import re
import subprocess

import pytest
import torch

import zero_sharded_mixed_flatten_amd as zs
from tests.test_lib_host import cpu_only
from tests.test_linear_host import BIG, EALIAS, EINVAL, L, ROOT, at


def test_every_declared_entry_point_is_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "zero_norm.h")).read()
    names = re.findall(r"^ZERO_API\s+[\w\s\*]*?\b(zero_\w+)\s*\(", src, flags=re.M)
    assert sorted(names) == ["zero_layernorm", "zero_layernorm_backward",
                             "zero_layernorm_workspace_bytes"]
    for n in names:
        assert hasattr(L, n) and callable(getattr(zs, n)) and n in zs.__all__


def test_the_header_is_plain_c(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "zero_norm.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"),
                    "-o", str(tmp_path / "s"), str(src)], check=True)


def test_workspace_sizes():
    assert zs.zero_layernorm_workspace_bytes(0, 1600) == 0
    assert zs.zero_layernorm_workspace_bytes(1600, 0) == 0
    for n in (1, 7, 4096, 16384, 16385, 1 << 20):
        sizes = [zs.zero_layernorm_workspace_bytes(m, n) for m in (1, 8, 600, 10000, BIG)]
        assert sizes == sorted(sizes) and sizes[0] >= 8 * n and sizes[-1] <= (1 << 16) * (n + 8)
    for bad in ((-1, 1), (1, -1), (BIG + 1, 1), (1, BIG + 1)):
        with pytest.raises(ValueError):
            zs.zero_layernorm_workspace_bytes(*bad)


FWD = dict(x=at(1), xdt=0, ldx=64, w=at(2), b=at(3), wdt=0, m=32, n=64, eps=1e-5, y=at(4), ydt=0,
           ldy=64, mean=at(5), rstd=at(6), stream=None)
BACK = dict(dy=at(1), dydt=0, lddy=64, x=at(2), xdt=0, ldx=64, w=at(3), wdt=0, mean=at(4),
            rstd=at(5), m=32, n=64, res=at(6), ldr=64, dx=at(7), lddx=64, dw=at(8), db=at(9),
            gdt=2, acc=0, ws=at(10), wsb=1 << 30, stream=None)
CALLS = {"fwd": (L.zero_layernorm, FWD), "back": (L.zero_layernorm_backward, BACK)}


def status(op, **change):
    fn, base = CALLS[op]
    return fn(*{**base, **change}.values())


@cpu_only
@pytest.mark.parametrize("op,change,want", [
    ("fwd", dict(wdt=2), EINVAL), ("fwd", dict(wdt=7), EINVAL), ("fwd", dict(xdt=1), EINVAL),
    ("fwd", dict(ydt=1), EINVAL), ("fwd", dict(xdt=-1), EINVAL), ("fwd", dict(m=-1), EINVAL),
    ("fwd", dict(n=BIG + 1, ldx=1 << 33, ldy=1 << 33), EINVAL), ("fwd", dict(ldx=63), EINVAL),
    ("fwd", dict(ldy=63), EINVAL), ("fwd", dict(x=None), EINVAL), ("fwd", dict(y=None), EINVAL),
    ("fwd", dict(x=at(1, 1)), EINVAL), ("fwd", dict(xdt=2, x=at(1, 2)), EINVAL),
    ("fwd", dict(w=at(2, 1)), EINVAL), ("fwd", dict(b=at(3, 1)), EINVAL),
    ("fwd", dict(mean=at(5, 2)), EINVAL), ("fwd", dict(rstd=at(6, 2)), EINVAL),
    ("fwd", dict(eps=0.0), EINVAL), ("fwd", dict(eps=-1.0), EINVAL),
    ("fwd", dict(eps=math.nan), EINVAL), ("fwd", dict(eps=math.inf), EINVAL),
    ("fwd", dict(eps=1e-60), EINVAL), ("fwd", dict(eps=1e60), EINVAL),
    ("fwd", dict(ldx=1 << 60), EINVAL), ("fwd", dict(n=0), EINVAL),
    ("fwd", dict(y=at(1, 2)), EALIAS), ("fwd", dict(y=at(1), ldy=65), EALIAS),
    ("fwd", dict(y=at(1), ydt=2), EALIAS), ("fwd", dict(y=at(2)), EALIAS),
    ("fwd", dict(y=at(3)), EALIAS), ("fwd", dict(y=at(5)), EALIAS), ("fwd", dict(y=at(6)), EALIAS),
    ("fwd", dict(mean=at(6)), EALIAS), ("fwd", dict(mean=at(1)), EALIAS),
    ("fwd", dict(rstd=at(2)), EALIAS), ("fwd", dict(rstd=at(3, 4)), EALIAS),
    ("back", dict(wdt=2), EINVAL), ("back", dict(xdt=1), EINVAL), ("back", dict(dydt=1), EINVAL),
    ("back", dict(gdt=1), EINVAL), ("back", dict(m=BIG + 1), EINVAL), ("back", dict(n=-1), EINVAL),
    ("back", dict(lddy=63), EINVAL), ("back", dict(ldx=63), EINVAL), ("back", dict(ldr=63), EINVAL),
    ("back", dict(lddx=63), EINVAL), ("back", dict(dy=None), EINVAL), ("back", dict(x=None), EINVAL),
    ("back", dict(dx=None), EINVAL), ("back", dict(mean=None), EINVAL),
    ("back", dict(rstd=None), EINVAL), ("back", dict(mean=at(4, 2)), EINVAL),
    ("back", dict(dw=at(8, 2)), EINVAL), ("back", dict(db=at(9, 1)), EINVAL),
    ("back", dict(res=at(6, 1)), EINVAL), ("back", dict(w=at(3, 1)), EINVAL),
    ("back", dict(ws=None), EINVAL), ("back", dict(ws=at(10, 8)), EINVAL),
    ("back", dict(wsb=64), EINVAL), ("back", dict(dw=None, ws=None), EINVAL),
    ("back", dict(dx=at(2)), EALIAS), ("back", dict(dx=at(3)), EALIAS),
    ("back", dict(dx=at(4)), EALIAS), ("back", dict(dx=at(5)), EALIAS),
    ("back", dict(dx=at(8)), EALIAS), ("back", dict(dx=at(9)), EALIAS),
    ("back", dict(dx=at(10)), EALIAS), ("back", dict(dx=at(1, 2)), EALIAS),
    ("back", dict(dx=at(1), lddx=65), EALIAS), ("back", dict(dx=at(1), dydt=2), EALIAS),
    ("back", dict(dx=at(6, 2)), EALIAS), ("back", dict(dx=at(6), lddx=70), EALIAS),
    ("back", dict(dw=at(1)), EALIAS), ("back", dict(dw=at(2)), EALIAS),
    ("back", dict(dw=at(3)), EALIAS), ("back", dict(db=at(4)), EALIAS),
    ("back", dict(db=at(6)), EALIAS), ("back", dict(db=at(8, 16)), EALIAS),
    ("back", dict(ws=at(1)), EALIAS), ("back", dict(ws=at(2)), EALIAS),
    ("back", dict(ws=at(3)), EALIAS), ("back", dict(ws=at(5)), EALIAS),
    ("back", dict(ws=at(6)), EALIAS), ("back", dict(ws=at(8)), EALIAS),
    ("back", dict(ws=at(9)), EALIAS)])
def test_refusals(op, change, want):
    assert status(op, **change) == want


@cpu_only
@pytest.mark.parametrize("op,change", [
    ("fwd", dict(m=0)), ("fwd", dict(n=0, mean=None, rstd=None)),
    ("fwd", dict(m=0, x=None, y=None, mean=None, rstd=None)), ("back", dict(n=0)),
    ("back", dict(m=0, dw=None, db=None, ws=None))])
def test_empty_outputs_are_no_ops(op, change):
    assert status(op, **change) == zs.ZERO_OK


def test_the_binding_refuses_what_is_not_a_gpu_matrix():
    x, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_layernorm(x, v, v, x)
    with pytest.raises(TypeError, match="GPU"):
        zs.zero_layernorm_backward(x, x, v, v, v, x)
