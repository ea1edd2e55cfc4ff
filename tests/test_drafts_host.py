"""The operators for drafted tokens without a GPU: refusals before any launch, trees, 8-bit weights."""
import math

import pytest
import torch

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
import test_decode_host as host  # noqa: E402

OK, INVALID, UNSUPPORTED, NO_DEVICE = 0, 1, 2, 3
BASE = host.BASE


@pytest.fixture(scope="module")
def h():
    d = decode.Decode(inspect_only=True)
    yield d.handle
    d.close()


def test_the_header_declares_them():
    assert {"mi_decode_rms_norm_f8", "mi_decode_f8_linear", "mi_decode_kv_append_at", "mi_decode_kv_attend_tree",
            "mi_decode_kv_keep", "mi_decode_kv_copy"} <= set(host.declared())


def norm(h, dtype=0, M=3, K=300, x=BASE, ldx=300, r=BASE << 1, ldr=300, g=BASE << 2, eps=1e-6, codes=BASE << 3, ldc=300,
         scales=BASE << 4, lds=3, total=BASE << 5, ldt=300):
    return decode._rms_norm_f8(h, dtype, M, K, x, ldx, r, ldr, g, eps, codes, ldc, scales, lds, total, ldt, None)


@pytest.mark.parametrize("change, status", [
    ({}, NO_DEVICE), (dict(g=None), NO_DEVICE), (dict(total=None), NO_DEVICE), (dict(r=None, total=None), NO_DEVICE),
    (dict(total=BASE), NO_DEVICE), (dict(total=BASE << 1), NO_DEVICE), (dict(eps=0.0), NO_DEVICE),
    (dict(M=0, x=None), OK), (dict(K=0, codes=None), OK),
    (dict(M=1, ldx=0, ldr=0, ldc=0, lds=0, ldt=0), NO_DEVICE),
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(r=None), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(ldx=299), INVALID), (dict(ldr=299), INVALID), (dict(ldc=299), INVALID), (dict(lds=2), INVALID), (dict(ldt=299), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(x=BASE + 1), UNSUPPORTED), (dict(scales=(BASE << 4) + 2), UNSUPPORTED),
    (dict(ldx=1 << 31), UNSUPPORTED), (dict(M=1 << 40), UNSUPPORTED), (dict(K=1 << 40, ldx=1 << 40), UNSUPPORTED),
    (dict(total=BASE, ldt=304), INVALID), (dict(total=BASE + 2), INVALID), (dict(codes=BASE + 100), INVALID),
    (dict(scales=(BASE << 2) + 4), INVALID), (dict(codes=(BASE << 5) + 1), INVALID), (dict(scales=(BASE << 3) + 896), INVALID),
    (dict(scales=(BASE << 3) + 900), NO_DEVICE),
])
def test_norm_arguments(h, change, status):
    assert norm(h, **change) == status
    assert norm(None, **change) == INVALID


def linear(h, dtype=0, M=3, N=300, K=200, x=BASE, ldx=200, xs=BASE << 1, ldxs=2, w=BASE << 2, ldw=200, ws=BASE << 3, ldws=2,
           b=BASE << 4, y=BASE << 5, ldy=300):
    return decode._f8_linear(h, dtype, M, N, K, x, ldx, xs, ldxs, w, ldw, ws, ldws, b, y, ldy, None)


@pytest.mark.parametrize("change, status", [
    ({}, NO_DEVICE), (dict(b=None), NO_DEVICE), (dict(M=0, x=None, y=None), OK), (dict(N=0, y=None), OK),
    (dict(K=0, x=None, w=None, xs=None, ws=None), NO_DEVICE), (dict(x=BASE + 1, w=(BASE << 2) + 3), NO_DEVICE),
    (dict(M=1, ldx=0, ldxs=0, ldy=0), NO_DEVICE), (dict(N=1, ldw=0, ldws=0, ldy=1), NO_DEVICE), (dict(N=128, ldws=0), NO_DEVICE),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(xs=None), INVALID), (dict(ws=None), INVALID), (dict(y=None), INVALID), (dict(ldx=199), INVALID), (dict(ldw=199), INVALID),
    (dict(ldxs=1), INVALID), (dict(ldws=1), INVALID), (dict(ldy=299), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(xs=(BASE << 1) + 2), UNSUPPORTED), (dict(ws=(BASE << 3) + 1), UNSUPPORTED), (dict(y=(BASE << 5) + 1), UNSUPPORTED),
    (dict(N=1 << 40), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(ldw=1 << 31), UNSUPPORTED),
    (dict(y=BASE + 590), INVALID), (dict(y=BASE + 600), NO_DEVICE), (dict(y=(BASE << 2) + 50000), INVALID),
    (dict(y=(BASE << 1) + 20), INVALID), (dict(y=(BASE << 3) + 4), INVALID), (dict(y=BASE << 4), INVALID),
])
def test_linear_arguments(h, change, status):
    assert linear(h, **change) == status
    assert linear(None, **change) == INVALID


def attend(h, cache=None, batch=None, dtype=0, max_len=100, hq=4, q=None, out=None, seen=BASE * 20, stride=1, words=1, scale=1.0,
           window=0, sinks=0):
    return decode._kv_attend_tree(h, host.ref(cache or host.cache_struct()), dtype, host.ref(batch or host.batch_struct()), max_len,
                                  hq, host.ref(q or host.rows(11, 4)), host.ref(out or host.rows(12, 4)), seen, stride, words, scale,
                                  window, sinks, None)


def test_attend_tree_arguments(h):
    for change, status in [
        ({}, NO_DEVICE), (dict(words=2, stride=3), NO_DEVICE), (dict(seen=None), INVALID), (dict(words=0, stride=0), INVALID),
        (dict(words=-1), INVALID), (dict(words=2, stride=1), INVALID), (dict(seen=BASE * 20 + 2), UNSUPPORTED),
        (dict(batch=host.batch_struct(tokens=90, max_tokens=33)), INVALID),
        (dict(batch=host.batch_struct(tokens=90, max_tokens=33), words=2, stride=2), NO_DEVICE),
        (dict(batch=host.batch_struct(tokens=0), seen=None), OK), (dict(hq=3), INVALID), (dict(scale=math.nan), INVALID),
        (dict(window=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(q=host.rows(12, 4)), INVALID),
        *[(dict(cache=host.cache_struct(**c)), st) for c, st in host.CACHE_FAULTS],
        *[(dict(batch=host.batch_struct(**c)), st) for c, st in host.BATCH_FAULTS],
    ]:
        assert attend(h, **change) == status, change
        assert attend(None, **change) == INVALID


def test_append_at_arguments(h):
    def call(positions=BASE * 20, rope=BASE * 8, rope_rows=3, rot=64):
        return decode._kv_append_at(h, host.ref(host.cache_struct()), 0, host.ref(host.batch_struct()), host.ref(host.rows(9, 2)),
                                    host.ref(host.rows(10, 2)), rope, rope_rows, rot, 0, positions, 4, host.ref(host.rows(11, 4)),
                                    host.ref(host.rows(12, 4)), None)
    assert call() == NO_DEVICE
    assert call(positions=None) == INVALID  # then the rows have to reach the table's last position
    assert call(positions=None, rope_rows=128) == NO_DEVICE
    assert call(rope_rows=0) == INVALID
    assert call(positions=BASE * 20 + 1) == UNSUPPORTED
    assert call(rot=24) == UNSUPPORTED


def test_keep_and_copy_arguments(h):
    def kept(handle=h, cache=None, batch=None, keep=BASE * 20):
        return decode._kv_keep(handle, host.ref(cache or host.cache_struct()), host.ref(batch or host.batch_struct()), keep, None)

    def copy(handle=h, cache=None, src=BASE * 20, dst=BASE * 21, pairs=3):
        return decode._kv_copy(handle, host.ref(cache or host.cache_struct()), src, dst, pairs, None)

    assert kept() == copy() == NO_DEVICE
    assert kept(None) == copy(None) == INVALID
    assert kept(keep=None) == copy(src=None) == copy(dst=None) == copy(pairs=-1) == INVALID
    assert kept(keep=BASE + 2) == copy(src=BASE + 1) == copy(dst=BASE + 2) == UNSUPPORTED
    assert copy(pairs=0, src=None) == copy(cache=host.cache_struct(pages=0)) == OK
    assert kept(batch=host.batch_struct(tokens=0), keep=None) == OK
    for change, status in host.CACHE_FAULTS:
        assert kept(cache=host.cache_struct(**change)) == copy(cache=host.cache_struct(**change)) == status
    for change, status in host.BATCH_FAULTS:
        assert kept(batch=host.batch_struct(**change)) == status
    assert decode._kv_keep(h, None, host.ref(host.batch_struct()), BASE, None) == decode._kv_copy(h, None, BASE, BASE, 1, None) == INVALID


def test_trees():
    seen, depth = decode.tree([-1, 0, 0, 2, -1, 4])
    assert seen.tolist() == [[1], [3], [5], [13], [16], [48]] and depth.tolist() == [0, 1, 1, 2, 0, 1]
    seen, depth = decode.tree(torch.arange(-1, 69))
    assert seen.shape == (70, 3) and seen.dtype == depth.dtype == torch.int32 and depth.tolist() == list(range(70))
    for i in range(70):
        assert [int(seen[i, w]) & 0xffffffff for w in range(3)] == [(2 ** (i + 1) - 1) >> 32 * w & 0xffffffff for w in range(3)]
    seen, depth = decode.tree([])
    assert seen.shape == (0, 0) and depth.shape == (0,)
    for bad in ([0], [-1, 1], [-2], [-1, 5]):
        with pytest.raises(ValueError):
            decode.tree(bad)


def test_eight_bit_weights():
    gen = torch.Generator().manual_seed(1)
    w = torch.randn((200, 300), generator=gen) * 0.1
    w[:128, 128:256] = 0
    w[130, 5] = 40.0
    q = decode.f8_quantize(w)
    assert q.weight.shape == (200, 300) and q.weight.dtype == torch.float8_e4m3fn and q.weight.is_contiguous()
    assert q.scales.shape == (2, 3) and q.scales[0, 1] == 0 and abs(float(q.scales[1, 0]) - 40 / 448) < 1e-7
    back = decode.f8_values(q.weight, q.scales)
    s = q.scales.repeat_interleave(128, 0)[:200].repeat_interleave(128, 1)[:, :300]
    # half a step of a code, or of the smallest; the quotient and the product are rounded too
    assert torch.all((back - w).abs() <= torch.maximum(w.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20))
    assert float(back[130, 5]) == pytest.approx(40.0, rel=2.0 ** -22)
    w[3, 4] = math.nan
    q = decode.f8_quantize(w)
    assert torch.isnan(decode.f8_values(q.weight, q.scales)[3, 4]) and torch.isfinite(decode.f8_values(q.weight, q.scales)[128:]).all()
    rows = decode.f8_values(q.weight[:5], torch.ones((5, 3)))
    assert rows.shape == (5, 300)
    for bad in (w[0], w.int()):
        with pytest.raises(ValueError):
            decode.f8_quantize(bad)
    with pytest.raises(ValueError):
        decode.f8_values(q.weight, q.scales[:1])
