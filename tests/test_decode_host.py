"""libmi_decode without a GPU: exports, argument checks before any launch, the weight layout."""
import ctypes
import os
import re

import pytest
import torch

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mi_decode.h")
OK, INVALID, UNSUPPORTED, NO_DEVICE = 0, 1, 2, 3
BASE = 1 << 40  # stands for device addresses: nothing here is ever followed


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mi_decode_\w+)\s*\(", text)))


def test_exports_every_declared_symbol():
    L = ctypes.CDLL(decode.LIB_PATH)
    assert {"mi_decode_w4_linear", "mi_decode_kv_append", "mi_decode_kv_read", "mi_decode_kv_attend"} <= set(declared())
    assert [n for n in declared() if not hasattr(L, n)] == []


@pytest.fixture(scope="module")
def h():
    d = decode.Decode(inspect_only=True)
    yield d.handle
    d.close()


def test_create_and_status_strings():
    assert decode._create(None, 1) == INVALID
    assert decode._destroy(None) == OK
    assert decode._status_string(2) == b"MI_DECODE_ERR_UNSUPPORTED"
    assert decode._status_string(99) == b"unknown status"
    assert decode._last_hip_error(None) == 0


def w4(h, dtype=0, M=3, N=40, K=256, group=128, x=BASE, ldx=None, qw=BASE << 1, sc=BASE << 2, z=None,
       bias=None, y=BASE << 3, ldy=None):
    return decode._w4_linear(h, dtype, M, N, K, group, x, K if ldx is None else ldx, qw, sc, z, bias, y,
                             N if ldy is None else ldy, None)


@pytest.mark.parametrize("change, status", [
    ({}, NO_DEVICE),
    (dict(bias=BASE << 4, z=BASE << 5), NO_DEVICE),
    (dict(M=0, x=None, y=None), OK),
    (dict(N=0, y=None), OK),
    (dict(K=0, x=None, qw=None, sc=None), NO_DEVICE),
    (dict(dtype=2), UNSUPPORTED),
    (dict(M=-1), INVALID),
    (dict(N=-1), INVALID),
    (dict(K=-1), INVALID),
    (dict(group=0), INVALID),
    (dict(group=48), UNSUPPORTED),
    (dict(ldx=255), INVALID),
    (dict(ldy=39), INVALID),
    (dict(M=1, ldx=0, ldy=0), NO_DEVICE),
    (dict(x=None), INVALID),
    (dict(y=None), INVALID),
    (dict(qw=None), INVALID),
    (dict(sc=None), INVALID),
    (dict(qw=(BASE << 1) + 8), UNSUPPORTED),
    (dict(x=BASE + 1), UNSUPPORTED),
    (dict(y=BASE + 2 * 3 * 256 - 2), INVALID),
    (dict(y=BASE + 2 * 3 * 256), NO_DEVICE),
    (dict(y=(BASE << 1) + 1024), INVALID),
    (dict(N=1 << 40), UNSUPPORTED),
])
def test_w4_arguments(h, change, status):
    assert w4(h, **change) == status
    assert w4(None, **change) == INVALID


def cache_struct(**kw):
    c = dict(k=BASE, v=BASE * 2, k_scale=BASE * 3, v_scale=BASE * 4, pages=10, kv_heads=2, page_size=32,
             head_dim=64, code=0)
    c.update(kw)
    return decode._Cache(**c)


def batch_struct(**kw):
    c = dict(table=BASE * 5, lens=BASE * 6, cu=BASE * 7, table_stride=4, table_cols=4, batch=3, tokens=9,
             max_tokens=5)
    c.update(kw)
    return decode._Batch(**c)


def rows(at, heads, D=64, ts=None, hs=None):
    return decode._Rows(None if at is None else BASE * at, heads * D if ts is None else ts, D if hs is None else hs)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(h, cache=None, batch=None, dtype=0, k=None, v=None, rope=BASE * 8, rope_rows=128, rot=64, hq=4,
           q=None, q_out=None):
    return decode._kv_append(h, ref(cache or cache_struct()), dtype, ref(batch or batch_struct()),
                             ref(k or rows(9, 2)), ref(v or rows(10, 2)), rope, rope_rows, rot, 0, hq,
                             ref(q or rows(11, 4)), ref(q_out or rows(12, 4)), None)


CACHE_FAULTS = [
    (dict(code=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(kv_heads=0), INVALID), (dict(pages=-1), INVALID), (dict(k=None), INVALID),
    (dict(v_scale=None), INVALID), (dict(v=BASE + 8), UNSUPPORTED),
]
BATCH_FAULTS = [
    (dict(batch=-1), INVALID), (dict(tokens=-1), INVALID), (dict(max_tokens=0), INVALID),
    (dict(table_stride=3), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(cu=None), INVALID), (dict(table_cols=1 << 27, table_stride=1 << 27), UNSUPPORTED),
]


@pytest.mark.parametrize("kw, status", CACHE_FAULTS)
def test_every_cache_call_checks_its_cache(h, kw, status):
    c = cache_struct(**kw)
    assert append(h, cache=c) == status
    assert attend(h, cache=c) == status
    assert decode._kv_read(h, ref(c), 0, ref(batch_struct()), BASE, BASE, None) == status


@pytest.mark.parametrize("kw, status", BATCH_FAULTS)
def test_every_cache_call_checks_its_batch(h, kw, status):
    t = batch_struct(**kw)
    assert append(h, batch=t, rope_rows=1 << 40) == status
    assert attend(h, batch=t) == status
    assert decode._kv_read(h, ref(cache_struct()), 0, ref(t), BASE, BASE, None) == status


@pytest.mark.parametrize("kw", [dict(batch=0), dict(tokens=0)])
def test_empty_batches_do_nothing(h, kw):
    t = batch_struct(**kw)
    assert append(h, batch=t) == OK
    assert attend(h, batch=t) == OK
    assert decode._kv_read(h, ref(cache_struct()), 0, ref(t), None, None, None) == OK


@pytest.mark.parametrize("kw, status", [
    ({}, NO_DEVICE),
    (dict(hq=0), NO_DEVICE),
    (dict(rope=None, rope_rows=0, rot=0), NO_DEVICE),
    (dict(rot=32), NO_DEVICE),
    (dict(rot=24), UNSUPPORTED),
    (dict(rot=80), INVALID),
    (dict(rope_rows=127), INVALID),
    (dict(dtype=3), UNSUPPORTED),
    (dict(hq=-1), INVALID),
    (dict(k=rows(None, 2)), INVALID),
    (dict(v=rows(10, 2, hs=63)), INVALID),
    (dict(k=rows(9, 2, ts=130)), UNSUPPORTED),
    (dict(q_out=rows(11, 4)), NO_DEVICE),                     # in place
    (dict(q_out=rows(11, 4, ts=512)), INVALID),               # over q, otherwise laid out
    (dict(q_out=rows(9, 4)), INVALID),                        # over k
])
def test_append_arguments(h, kw, status):
    assert append(h, **kw) == status
    assert append(None, **kw) == INVALID


def attend(h, cache=None, batch=None, dtype=0, max_len=128, hq=4, q=None, out=None, scale=0.1, window=0, sinks=0):
    return decode._kv_attend(h, ref(cache or cache_struct()), dtype, ref(batch or batch_struct()), max_len, hq,
                             ref(q or rows(11, 4)), ref(out or rows(12, 4)), scale, window, sinks, None)


@pytest.mark.parametrize("kw, status", [
    ({}, NO_DEVICE),
    (dict(window=5, sinks=2), NO_DEVICE),
    (dict(scale=0.0), NO_DEVICE),
    (dict(dtype=2), UNSUPPORTED),
    (dict(hq=3), INVALID),
    (dict(hq=0), INVALID),
    (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID),
    (dict(max_len=-1), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(out=rows(11, 4)), INVALID),
    (dict(q=rows(11, 4, ts=257)), UNSUPPORTED),
    (dict(out=rows(None, 4)), INVALID),
])
def test_attend_arguments(h, kw, status):
    assert attend(h, **kw) == status
    assert attend(None, **kw) == INVALID


@pytest.mark.parametrize("N, K, group", [(1, 1, 32), (16, 128, 32), (17, 129, 64), (40, 300, 128), (33, 96, 320)])
@pytest.mark.parametrize("with_zeros", [False, True])
def test_pack_and_unpack(N, K, group, with_zeros):
    g = torch.Generator().manual_seed(N * K)
    groups = -(-K // group)
    codes = torch.randint(0, 16, (N, K), generator=g)
    scales = torch.rand((N, groups), generator=g).half()
    zeros = torch.randint(0, 16, (N, groups), generator=g) if with_zeros else None
    w = decode.w4_pack(codes, scales, zeros, group)
    assert w.qweight.shape == (-(-N // 16), -(-K // 128), 64, 4) and w.scales.shape == (groups, -(-N // 16) * 16)
    col = torch.arange(K) // group
    want = (codes - (8 if zeros is None else zeros[:, col])).float() * scales.float()[:, col]
    assert torch.equal(decode.w4_unpack(w), want)
    # the layout as the header states it, word by word
    for n, k in [(0, 0), (N - 1, K - 1), (N // 2, K // 3)]:
        e = k % 8
        word = int(w.qweight[n // 16, k // 128, (k % 32 // 8) * 16 + n % 16, k % 128 // 32]) & 0xFFFFFFFF
        assert word >> (4 * (e // 2) + 16 * (e % 2)) & 15 == int(codes[n, k])


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_is_within_half_a_step(symmetric):
    w = torch.randn((50, 200), generator=torch.Generator().manual_seed(3)).half()
    w[7] = 0
    p = decode.w4_quantize(w, 64, symmetric)
    step = p.scales.float().t()[:50, torch.arange(200) // 64]
    # half a step, and what rounding the scale to fp16 moves at most 15 steps by
    err = (decode.w4_unpack(p) - w.float()).abs()
    assert torch.all(err <= step * (0.5 + 16 * 2.0 ** -11 + (0.5 if not symmetric else 0)))
    assert torch.all(decode.w4_unpack(p)[7] == 0)


def test_pack_refuses():
    c, s = torch.zeros((4, 64), dtype=torch.uint8), torch.ones((4, 1)).half()
    for bad in (dict(group=0), dict(group=40), dict(scales=torch.ones((4, 2)).half()), dict(codes=c[0]),
                dict(zeros=torch.zeros((4, 2)))):
        with pytest.raises(ValueError):
            decode.w4_pack(**{**dict(codes=c, scales=s, group=64), **bad})
    with pytest.raises(TypeError):
        decode.w4_pack(c, s.double(), group=64)


def test_wrappers_refuse_host_tensors():
    d = decode.Decode(inspect_only=True)
    w = decode.w4_quantize(torch.randn(16, 64).half(), 64)
    with pytest.raises(ValueError):
        d.w4_linear(torch.zeros((1, 64)).half(), w.qweight, w.scales, n=16, group=64)
    with pytest.raises(TypeError):
        d.w4_linear(torch.zeros((1, 64)), w.qweight, w.scales, n=16, group=64)
    with pytest.raises(ValueError):
        decode.KvCache.empty(2, 1, 64, device="cpu")
