"""The products' direct copies as compiled (CPU).  The copy instruction is
written out, so the compiler does not keep its distances: it must follow the
write of m0 by one wait state, and a vector write of the scalar registers that
hold its address (a spilled register's way back) by five."""
import os
import re

import pytest

isa = pytest.importorskip("tests.test_lib_isa")
SOURCE = os.path.join(isa.CSRC, "linear.hip")
needs_hipcc = pytest.mark.skipif(not os.path.exists(isa.HIPCC), reason="hipcc not available")


@needs_hipcc
def test_every_copy_carries_its_wait_states():
    copies = 0
    for block in isa._inline_asm_blocks(isa._asm(SOURCE)):
        for i, line in enumerate(block):
            if "global_load_lds" not in line:
                continue
            copies += 1
            m = isa.NOP.match(block[i - 1]) if i else None
            assert m and int(m.group(1)) >= 4, f"{line.strip()!r} in {block}"
    assert copies > 0


@needs_hipcc
def test_m0_is_written_by_the_scalar_unit_and_read_by_the_copies_only():
    """the compiler itself puts each copy's address into m0 (an input of the
    statement, not one of its own writes), and nothing else uses the register"""
    asm = isa._asm(SOURCE)
    blocks = isa._inline_asm_blocks(asm)
    assert not any("m0" in line for b in blocks for line in b)
    uses = [line for line in asm.splitlines() if re.search(r"\bm0\b", line.split(";")[0])]
    assert uses
    for line in uses:
        assert re.match(r"^\s*s_\w+\s+m0,", line) and line.count("m0") == 1, line
