"""Device code of the operators for drafted tokens, without a GPU: what hand-written copies into shared memory have to wait for."""
import re
import subprocess

import pytest

from test_decode_device_code import LLVM, code_objects  # noqa: F401  (a fixture)

REGISTERS = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")


def scalars(text):
    out = set()
    for lo, hi, one in REGISTERS.findall(text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def states(ins):
    """Wait states that an instruction is."""
    return int(ins.split()[1], 0) + 1 if ins.startswith("s_nop") else 1


def early_copies(listing):
    """Copies from memory into shared memory that come too early: one wait state lies between a write of m0 and the
    copy that reads it, and five between a vector instruction's scalar result and the copy that takes it."""
    bad, copies, before = [], 0, []
    for ins in listing:
        if ins.endswith(":"):
            before = []
            continue
        op = ins.split()[0]
        if op.startswith("buffer_load") and ins.endswith(" lds"):
            copies += 1
            passed = 0
            for old in reversed(before[-6:]):
                what = old.split()[0]
                if passed < 1 and re.match(r"s_\S+ m0\b", old):
                    bad.append((old, ins))
                written = scalars(old.split(",")[0]) if what.startswith("v_") else set()
                if passed < 5 and written & scalars(ins):
                    bad.append((old, ins))
                passed += states(old)
        before.append(ins)
    return copies, bad


def listing(co):
    text = subprocess.run([LLVM + "/llvm-objdump", "-d", str(co)], check=True, capture_output=True, text=True).stdout
    for line in text.splitlines():
        if re.match(r"[0-9a-f]+ <", line):
            yield "function:"
        elif line.startswith("\t"):
            yield re.sub(r"\s+", " ", line.split("//")[0]).strip()


def test_planted_mistakes_are_found():
    copy = "buffer_load_dwordx4 v1, s[8:11], s14 offen lds"
    assert early_copies(["s_add_u32 m0, s1, s2", copy])[1]
    assert early_copies(["s_mov_b32 m0, s1", copy])[1]
    assert not early_copies(["s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert not early_copies(["s_mov_b32 m0, s1", "v_add_u32_e32 v2, v3, v4", copy])[1]
    assert early_copies(["v_readfirstlane_b32 s14, v2", "s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert early_copies(["v_readfirstlane_b32 s9, v2", "s_nop 2", "s_nop 0", copy])[1]
    assert not early_copies(["v_readfirstlane_b32 s9, v2", "s_nop 3", "s_nop 0", copy])[1]
    assert not early_copies(["v_readfirstlane_b32 s15, v2", "s_mov_b32 m0, s1", "s_nop 0", copy])[1]
    assert early_copies([copy, copy]) == (2, [])


def test_copies_into_shared_memory_wait_for_what_they_read(code_objects):  # noqa: F811
    copies, bad = 0, []
    for co in code_objects:
        n, early = early_copies(listing(co))
        copies, bad = copies + n, bad + early
    if copies == 0:
        pytest.fail("no copies found")
    assert not bad, (len(bad), bad[:5])
