"""Wait states in the built library's gfx950 code (CPU): between a vector instruction
that writes a register and a lane swap (v_permlane16_swap, v_permlane32_swap) or a
DPP operand that reads it there are two wait states.  The hardware does not wait for
either.  The compiler counts them where it sees both instructions, but not where one
of the two stands in inline assembly; this counts them in what it made."""
import os
import re
import struct
import subprocess

import pytest

import gated_delta_rule_ckda_amd as ck
from gated_delta_rule_ckda_amd import build as libbuild

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(libbuild.HIPCC)), "llvm", "bin", "llvm-objdump")
BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"
NEED = 2
DPP = re.compile(r"quad_perm:|row_(shl|shr|ror|mirror|half_mirror|bcast|newbcast|share|xmask)\b|wave_(shl|rol|shr|ror)\b")
REG = re.compile(r"^[|\-]*v(?:(\d+)|\[(\d+):(\d+)\])")


def code_objects(path):
    """The gfx950 code objects of a library: a bundle is its mark, a count, and for each entry offset, size and name."""
    with open(path, "rb") as f:
        data = f.read()
    out, i = [], data.find(BUNDLE)
    while i >= 0:
        count, = struct.unpack_from("<Q", data, i + len(BUNDLE))
        p = i + len(BUNDLE) + 8
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, p)
            if data[p + 24:p + 24 + name].endswith(b"gfx950"):
                out.append(data[i + offset:i + offset + size])
            p += 24 + name
        i = data.find(BUNDLE, i + len(BUNDLE))
    return out


def registers(operand):
    m = REG.match(operand)
    if not m:
        return range(0)
    first = int(m.group(1) or m.group(2))
    return range(first, int(m.group(3) or first) + 1)


def places(text):
    """(instruction, register, wait states) of every lane swap and DPP operand that reads too early, and the count of
    those that were looked at.  `text`: one code object as llvm-objdump writes it."""
    code, at, jumps, kernel = [], {}, {}, ""
    for line in text.splitlines():
        if line.endswith(">:"):
            kernel = line[line.index("<") + 1:-2]
            at[kernel] = int(line.split()[0], 16)
        if not line.startswith("\t") or "//" not in line:   # (padding behind a kernel is "...")
            continue
        ins, _, note = line.partition("//")
        name, _, rest = ins.strip().partition(" ")
        at[int(note[:note.index(":")], 16)] = len(code)
        if name.startswith("s_cbranch") or name == "s_branch":
            target = re.search(r"<(\S+?)(?:\+0x([0-9a-f]+))?>", note)
            jumps.setdefault(at[target.group(1)] + int(target.group(2) or "0", 16), []).append(len(code))
        code.append((name, rest, kernel))

    def before(i):
        """The instructions that may run just before i."""
        if i and code[i - 1][0] not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            yield i - 1
        yield from came.get(i, ())

    came = {at[target]: who for target, who in jumps.items()}

    def waits(i, reg):
        """Wait states since the last vector write of reg, or NEED if there are as many."""
        least, todo = NEED, [(j, 0) for j in before(i)]
        while todo:
            j, n = todo.pop()
            name, rest, _ = code[j]
            if name.startswith("v_") and not name.startswith(("v_mfma", "v_smfmac", "v_cmp", "v_readlane", "v_readfirstlane")):
                written = [o.strip() for o in rest.split(",")][:2 if "swap" in name else 1]
                if any(reg in registers(o) for o in written):
                    least = min(least, n)
                    continue
            n += int(rest, 0) + 1 if name == "s_nop" else 1
            if n < least:
                todo += [(k, n) for k in before(j)]
        return least

    bad, looked = [], 0
    for i, (name, rest, kernel) in enumerate(code):
        swap = name.startswith("v_permlane") and "swap" in name
        if not swap and not (name.startswith("v_") and DPP.search(rest)):
            continue
        operands = [o.strip() for o in rest.split(",")]
        for o in operands[:2] if swap else operands[1:2]:
            for reg in registers(o):
                looked += 1
                n = waits(i, reg)
                if n < NEED:
                    bad.append((kernel, f"{name} {rest.strip()}", f"v{reg}", n))
    return bad, looked


HEAD = "0000000000001000 <kernel>:\n"


def listing(*lines):
    return HEAD + "".join(f"\t{ins} // {0x1000 + 4 * i:012X}: 00000000{note}\n" for i, (ins, note) in
                          enumerate(x if isinstance(x, tuple) else (x, "") for x in lines))


@pytest.mark.parametrize("between,waits", [((), 0), (("s_nop 0",), 1), (("v_mul_f32_e32 v9, v8, v8",), 1), (("s_nop 1",), None),
                                           (("s_nop 0", "v_mul_f32_e32 v9, v8, v8"), None)])
def test_the_count_itself(between, waits):
    for reader, regs in (("v_permlane32_swap_b32_e32 v4, v5", ("v5",)), ("v_add_f32_dpp v1, v5, v6 row_ror:8 row_mask:0xf bank_mask:0xf", ("v5",)),
                         ("v_permlane16_swap_b32_e32 v5, v4", ("v5",))):
        bad, looked = places(listing("v_add_f32_e32 v5, v1, v2", *between, reader))
        assert looked == (2 if "swap" in reader else 1)
        assert [(b[2], b[3]) for b in bad] == ([] if waits is None else [(r, waits) for r in regs])


def test_the_count_follows_jumps():
    """The writer is the last instruction of a loop whose first one reads."""
    bad, _ = places(listing("v_mov_b32_e32 v5, 0", "s_nop 1", "v_mov_b32_dpp v1, v5 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf",
                            "v_add_f32_e32 v5, v1, v1", ("s_cbranch_scc1 65533", " <kernel+0x8>"), "s_endpgm"))
    assert [(b[2], b[3]) for b in bad] == [("v5", 1)]
    assert places(listing("v_mov_b32_e32 v5, 0", ("s_branch 1", " <kernel+0xc>"), "v_mov_b32_dpp v1, v5 row_mirror row_mask:0xf bank_mask:0xf",
                          "s_endpgm"))[0] == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not installed")
def test_lane_swaps_and_dpp_operands_wait_for_their_registers(tmp_path):
    if not os.path.exists(ck.LIB_PATH):
        libbuild.build()
    objects = code_objects(ck.LIB_PATH)
    assert objects
    total, bad = 0, []
    for i, data in enumerate(objects):
        path = tmp_path / f"{i}.elf"
        path.write_bytes(data)
        text = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
        wrong, looked = places(text)
        bad += wrong
        total += looked
    assert total > 10000
    assert not bad, (len(bad), bad[:5])
