"""The MXFP4 tile kernel issues its scaled MFMAs from inline asm, so the compiler's hazard recogniser does not see them.
This checks the built gfx950 code objects: no VALU instruction (a move, an AGPR write) that writes one of an MFMA's
source registers stands less than two wait states before it, and nothing reads or overwrites an MFMA's result by
VALU within the 18 wait states of its latency unless waits stand between (the kernel's epilogue begins with 24)."""

import os
import re
import shutil
import subprocess

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


def parse(listing):
    """(mnemonic, operands, places that control may come from) of a disassembly's instructions, symbol by symbol."""
    ins, at, jumps, header = [], {}, [], True
    base = {}
    for line in listing.splitlines():
        m = re.match(r"([0-9a-f]+) <(.+)>:$", line)
        if m:
            base[m[2]], header = int(m[1], 16), True
        m = re.match(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+): .*?(?:<(.+)\+0x([0-9a-f]+)>)?$", line)
        if not m:
            continue
        i = len(ins)
        at[int(m[3], 16)] = i
        through = not header and not ins[-1][0].startswith(("s_branch", "s_endpgm", "s_setpc"))
        ins.append((m[1], m[2], [i - 1] if through else []))
        header = False
        if m[1].startswith(("s_branch", "s_cbranch")):
            assert m[4] is not None, line
            jumps.append((i, base[m[4]] + int(m[5], 16)))
    for i, target in jumps:
        ins[at[target]][2].append(i)
    return ins


def late_writes(ins):
    """Scaled MFMAs with a source register that a VALU instruction writes less than two wait states before, on any path."""
    seen, bad = 0, []
    for i, (mn, ops, before) in enumerate(ins):
        if not mn.startswith("v_mfma_scale_f32_32x32x64"):
            continue
        seen += 1
        sources = registers(", ".join(split(ops)[1:]))
        todo = [(k, 0) for k in before]
        while todo:
            k, waits = todo.pop()
            m, o, b = ins[k]
            if m == "s_nop":
                waits += int(o.split()[0], 0) + 1
            else:
                if m.startswith("v_") and not m.startswith(("v_mfma", "v_cmp")) and registers(split(o)[0]) & sources:
                    bad.append((i, k, f"{m} {o} feeds {mn} {ops} after {waits} wait states"))
                waits += 1
            if waits < 2:
                todo += [(n, waits) for n in b]
    return seen, bad


def test_a_late_write_is_found():
    """The search itself, on a loop whose last move feeds the MFMA at its head, and on the same with waits."""
    mfma = "v_mfma_scale_f32_32x32x64_f8f6f4 a[0:15], v[0:3], v[4:7], a[0:15], v8, v9 op_sel_hi:[0,0,0] cbsz:4 blgp:4"

    def listing(wait):
        lines = ["v_mov_b32_e32 v8, 0", "s_nop 1", mfma, "v_mov_b32_e32 v9, v10"] + wait + ["s_cbranch_scc1 65000"]
        rows = [f"\t{x}  // {0x100 + 4 * i:012X}: 00000000" for i, x in enumerate(lines)]
        rows[-1] += " <k+0x8>"
        return "0000000000000100 <k>:\n" + "\n".join(rows)

    assert late_writes(parse(listing([])))[1] and late_writes(parse(listing([])))[0] == 1
    assert late_writes(parse(listing(["s_nop 0"])))[1] == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs llvm-objdump")
def test_no_late_write_on_any_path(tmp_path):
    """As the first test, following branches too (the head of the loop over K comes after its end)."""
    if not os.path.exists(LIB):
        pytest.skip("libfp8bq.so not built")
    shutil.copy(LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    seen = 0
    for o in sorted(f for f in os.listdir(tmp_path) if f.endswith("gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", o], cwd=tmp_path, check=True, capture_output=True,
                              text=True).stdout
        n, bad = late_writes(parse(text))
        seen += n
        assert not bad, bad[0][2]
    assert seen > 0
