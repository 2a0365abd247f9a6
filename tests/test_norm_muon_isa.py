"""The layer norm's and the Muon step's kernels as compiled (CPU): the
instruction forms that the library's other sources rule out are absent, the
products copy straight to shared memory and spill nothing, and their copies
carry their wait states."""
import os
import re

import pytest

isa = pytest.importorskip("tests.test_lib_isa")
from tests.test_linear_isa import _kernels  # noqa: E402

SOURCES = [os.path.join(isa.CSRC, f) for f in ("norm.hip", "muon.hip", "orthogonalize.hip")]
needs_hipcc = pytest.mark.skipif(not os.path.exists(isa.HIPCC), reason="hipcc not available")


@needs_hipcc
@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_forbidden_forms(src):
    asm = isa._asm(src)
    assert len(re.findall(r"^\s*\.amdhsa_kernel\b", asm, flags=re.M)) > 0
    # the elementwise steps round each operation; the norm and the products
    # round their outputs from fp32 and may use any fused form
    forms = isa.FORBIDDEN if "muon" in src else [f for f in isa.FORBIDDEN if "pk" in f]
    for pat in forms + isa.SCALAR_WRITES:
        hits = re.findall(pat + r"[^\n]*", asm)
        assert not hits, f"{src}: {len(hits)} x {hits[0]}"


@needs_hipcc
def test_wide_inline_stores_carry_their_wait_states():
    for block in isa._inline_asm_blocks(isa._asm(SOURCES[1])):
        for i, line in enumerate(block):
            if isa.WIDE_STORE.match(line):
                m = isa.NOP.match(block[i + 1]) if i + 1 < len(block) else None
                assert m and int(m.group(1)) >= 1, block


@needs_hipcc
def test_the_products():
    asm = isa._asm(SOURCES[2])
    seen = 0
    for name, body, tail in _kernels(asm):
        if not any(k in name for k in ("product_kernel", "small_kernel", "narrow_kernel")):
            continue
        assert re.search(r"; ScratchSize: (0|24)\b", tail), name  # 24: a row's broken end
        if "product_kernel" not in name or "Lb1E" in name:  # Lb1: joins parts
            continue
        seen += 1
        assert re.search(r"\bv_mfma_f32_16x16x32_f16\b", body)
        assert "global_load_lds_dwordx4" in body
        assert re.search(r"; ScratchSize: 0\b", tail), name
    assert seen >= 6
    copies = 0
    for block in isa._inline_asm_blocks(asm):
        assert not any("m0" in line for line in block)
        for i, line in enumerate(block):
            if "global_load_lds" in line:
                copies += 1
                m = isa.NOP.match(block[i - 1]) if i else None
                assert m and int(m.group(1)) >= 4, block
    assert copies > 0
    for line in asm.splitlines():
        if re.search(r"\bm0\b", line.split(";")[0]):
            assert re.match(r"^\s*s_\w+\s+m0,", line) and line.count("m0") == 1, line


@needs_hipcc
def test_the_norm_spills_nothing():
    for name, body, tail in _kernels(isa._asm(SOURCES[0])):
        assert re.search(r"; ScratchSize: 0\b", tail), name
