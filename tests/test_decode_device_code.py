"""Device code of libmi_decode, without a GPU: what its sources and its gfx950 code must hold."""
import glob
import os
import re

import test_asm_clobbers as clobbers

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
