"""The MXFP4 tile kernel issues its scaled MFMAs from inline asm, so the compiler's hazard recogniser does not see them.
This checks the built gfx950 code objects: no VALU instruction (a move, an AGPR write) that writes one of an MFMA's
source registers stands less than two wait states before it, and nothing reads or overwrites an MFMA's result by
VALU within the 18 wait states of its latency unless waits stand between (the kernel's epilogue begins with 24)."""

import os
import re

import pytest

from tests.test_lds_dma_m0 import OBJDUMP, PKG, _instructions

LIB = os.path.join(PKG, "libfp8bq.so")


def registers(text):
    """{'v12', 'a3', ...} named by an operand string."""
    out = set()
    for kind, a, b in re.findall(r"\b([va])\[(\d+):(\d+)\]", text):
        out |= {f"{kind}{i}" for i in range(int(a), int(b) + 1)}
    out |= {k + n for k, n in re.findall(r"\b([va])(\d+)\b", text)}
    return out


def split(ops):
    """Operands of an instruction, brackets kept together."""
    return [p.strip() for p in re.split(r",(?![^\[]*\])", ops)]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")
def test_no_valu_write_just_before_an_asm_mfma(tmp_path):
    if not os.path.exists(LIB):
        pytest.skip("libfp8bq.so not built")
    seen = 0
    for obj, ins in _instructions(LIB, tmp_path):
        for i, (mn, ops) in enumerate(ins):
            if not mn.startswith("v_mfma_scale_f32_32x32x64"):
                continue
            seen += 1
            parts = split(ops)
            dst, sources = registers(parts[0]), registers(", ".join(parts[1:]))
            waits, k = 0, i - 1
            while waits < 2 and k >= 0:
                m, o = ins[k]
                if m == "<label>":
                    break
                if m == "s_nop":
                    waits += int(o.split()[0], 0) + 1
                else:
                    if m.startswith("v_") and not m.startswith("v_mfma") and not m.startswith("v_cmp"):
                        wrote = registers(split(o)[0])
                        assert not wrote & sources, f"{obj} #{i}: {m} {o} feeds {mn} {ops} after {waits} wait states"
                    waits += 1
                k -= 1
            # results: an AGPR read or write of dst too soon after
            waits, k = 0, i + 1
            while waits < 18 and k < len(ins):
                m, o = ins[k]
                if m == "<label>" or m.startswith("s_cbranch") or m == "s_branch" or m == "s_endpgm":
                    break
                if m == "s_nop":
                    waits += int(o.split()[0], 0) + 1
                else:
                    if m.startswith("v_") and not m.startswith("v_mfma"):
                        assert not registers(o) & dst, f"{obj} #{k}: {m} {o} touches the result of {ops} after {waits} wait states"
                    waits += 1
                k += 1
    assert seen > 0, "no scaled MFMA found: the disassembly format changed?"
