"""Device code of libmi_decode, without a GPU: what its sources and its gfx950 code must hold."""
import glob
import os
import re
import shutil
import struct
import subprocess

import pytest

import test_asm_clobbers as clobbers

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
LLVM = "/opt/rocm/lib/llvm/bin"

HERE = os.path.dirname(os.path.abspath(__file__))
DECODE = os.path.join(HERE, "..", "dense_fp16_gemm_hgemm_amd", "decode")


def code(name):
    """A source file without its comments."""
    text = open(os.path.join(DECODE, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_a_waves_piece_of_shared_memory_is_ordered():
    """What one lane stores and another loads has an order that the compiler knows, in both directions."""
    text = code("w4.hip")
    events = []
    for m in re.finditer(r"(?P<sync>wave_shared\(\);)|(?P<store>\bxs\[[^;=]*\] = )|(?P<load>= xs\[)", text):
        events.append(m.lastgroup)
    # the rows that no load fills are cleared; then, for each block: store, order, load, order
    assert events == ["store", "store", "sync", "load", "sync"]
    body = text[text.index("inline void wave_shared()"):]
    assert '__builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");' in body[:200]
    assert "__builtin_amdgcn_wave_barrier();" in body[:200]


def test_inline_asm_declares_what_it_changes():
    for path in sorted(glob.glob(os.path.join(DECODE, "*.hip")) + glob.glob(os.path.join(DECODE, "*.hpp"))):
        for template, declared in clobbers.asm_statements(code(os.path.basename(path))):
            assert not clobbers.undeclared(template, declared), (path, template)


@pytest.fixture(scope="module")
def code_objects(tmp_path_factory):
    """The gfx950 code objects of libmi_decode, one for each source."""
    if not all(map(shutil.which, ("objcopy", LLVM + "/llvm-readelf", LLVM + "/llvm-objdump"))):
        pytest.skip("binutils or ROCm's LLVM tools are missing")
    folder = tmp_path_factory.mktemp("decode")
    fat = folder / "fat.bin"
    subprocess.run(["objcopy", "--dump-section", f".hip_fatbin={fat}", decode.LIB_PATH, str(folder / "copy.so")], check=True)
    data, found, at = fat.read_bytes(), [], 0
    while (at := data.find(b"__CLANG_OFFLOAD_BUNDLE__", at)) >= 0:
        count, pos = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, pos)
            name = data[pos + 24:pos + 24 + length].decode()
            pos += 24 + length
            if name.endswith("gfx950"):
                found.append(folder / f"{len(found)}.co")
                found[-1].write_bytes(data[at + offset:at + offset + size])
        at += 24
    assert len(found) >= 5
    return found


def test_no_array_is_left_in_scratch_memory(code_objects):
    """A few spilled registers (48 rows of 128 channels) take 44 bytes; an array of operands takes hundreds."""
    seen = {}
    for co in code_objects:
        notes = subprocess.run([LLVM + "/llvm-readelf", "--notes", "-W", str(co)], check=True, capture_output=True,
                               text=True).stdout
        for block in re.split(r"\n\s*- \.", notes):
            name = re.search(r"\.name:\s+(_ZN3mid\S+kernel\S*)", "." + block)
            if name:
                seen[name.group(1)] = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1))
    for kernel in ("attend_kernel", "attend_tile_kernel", "join_kernel", "w4_kernel", "w4_short_kernel", "append_kernel",
                   "read_kernel"):
        assert any(kernel in name for name in seen), kernel
    assert {n: b for n, b in seen.items() if b > 64} == {}


def test_no_packed_fp32_instructions(code_objects):
    for co in code_objects:
        text = subprocess.run([LLVM + "/llvm-objdump", "-d", str(co)], check=True, capture_output=True, text=True).stdout
        assert "v_mfma" in text or "global_load" in text or "buffer_load" in text
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
