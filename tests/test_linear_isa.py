"""The layer products' and the dropout's kernels as compiled (CPU): none of
the instruction forms that the library's other sources rule out, matrix
instructions and direct copies where they are meant to be, and no register
of the main loops spilled to memory."""
import os
import re

import pytest

isa = pytest.importorskip("tests.test_lib_isa")
SOURCES = [os.path.join(isa.CSRC, f) for f in ("linear.hip", "dropout.hip")]
needs_hipcc = pytest.mark.skipif(not os.path.exists(isa.HIPCC), reason="hipcc not available")


@needs_hipcc
@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_forbidden_forms(src):
    asm = isa._asm(src)
    assert len(re.findall(r"^\s*\.amdhsa_kernel\b", asm, flags=re.M)) > 0
    for pat in isa.FORBIDDEN + isa.SCALAR_WRITES:
        hits = re.findall(pat + r"[^\n]*", asm)
        assert not hits, f"{src}: {len(hits)} x {hits[0]}"


def _kernels(asm):
    """(name, body, resources) of every kernel"""
    for m in re.finditer(r"^(_Z\w+):\s*;\s*@", asm, flags=re.M):
        end = asm.index(".Lfunc_end", m.start())
        nxt = re.search(r"^_Z\w+:\s*;\s*@", asm[end:], flags=re.M)
        yield m.group(1), asm[m.start():end], asm[end:end + nxt.start()] if nxt else asm[end:]


@needs_hipcc
def test_the_tile_kernels_main_loops():
    seen = 0
    for name, body, tail in _kernels(isa._asm(SOURCES[0])):
        if "tile_kernel" not in name:
            continue
        seen += 1
        assert re.search(r"\bv_mfma_f32_16x16x32_(bf16|f16)\b", body)
        flags = re.findall(r"Lb([01])E", name)
        assert ("global_load_lds_dwordx4" in body) == (flags[-2] == "1")
        assert re.search(r"; ScratchSize: 0\b", tail), name
    assert seen >= 24
