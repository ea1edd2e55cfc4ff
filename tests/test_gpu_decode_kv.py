"""Appending to the paged 8-bit cache and reading it back, against the definition in float64."""
import pytest
import torch

from decode_ref import F, QMAX, half_step, layout, random_codes, rotate, values

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
DEV = torch.device("cuda", 0)
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


def put(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(past, new, H, D, page, codes, seed, spare=2, extra_cols=0):
    total = [p + n for p, n in zip(past, new)]
    pages = sum(-(-t // page) for t in total) + spare
    table = layout(total, page, pages, torch.Generator().manual_seed(seed), extra_cols)
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (pages, H, page, D)
    cache = decode.KvCache(random_codes(shape, codes, g), random_codes(shape, codes, g),
                           *[torch.rand((pages, H), generator=g, device=DEV) * 0.01 + 0.02 for _ in range(2)])
    if codes == torch.float8_e4m3fn:
        cache.k_scale.mul_(127 / 448)
        cache.v_scale.mul_(127 / 448)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cache, table, cu, g


def code_slip(x, s, codes):
    """How far a stored value may be from x (in units of the value) at scale s: half a step."""
    if codes == torch.int8:
        return s * 0.5
    return torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)  # normal codes; the subnormal step is 2^-9


def check_store(cache, was, was_scale, now, now_scale, x, table, past, new, cu):
    """Codes and scales after x [T, H, D] (float64) was appended: every touched slot, and the rest unchanged."""
    ps, codes = cache.page_size, cache.k.dtype
    raw_was, raw = was.view(torch.uint8), now.view(torch.uint8)
    same = torch.ones((cache.pages, ps), dtype=torch.bool, device=DEV)
    same_scale = torch.ones(cache.pages, dtype=torch.bool, device=DEV)
    for b in range(len(past)):
        for lo in range(past[b] // ps * ps, past[b] + new[b], ps):
            page = int(table[b, lo // ps])
            i, j = max(lo, past[b]), min(lo + ps, past[b] + new[b])
            if j <= i:
                continue
            fill = i - lo
            part = x[cu[b] + i - past[b]:cu[b] + j - past[b]]  # [n, H, D]
            mine = part.abs().amax((0, 2)) / QMAX[codes]
            old = was_scale[page].to(F) if fill else torch.zeros_like(mine)
            want = torch.maximum(old, mine)
            got = now_scale[page].to(F)
            # the largest value carries the rotation's rounding, the division one more
            assert torch.all((got - want).abs() <= 4 * 2.0 ** -23 * want), (b, page)
            stored = values(now[page])[:, fill:fill + j - i].transpose(0, 1) * got[:, None]
            slip = code_slip(part, want[:, None], codes) + 2.0 ** -20 * want[:, None] * QMAX[codes]
            assert torch.all((stored - part).abs() <= slip), (b, page, float(((stored - part).abs() / slip).max()))
            if fill:
                before = values(was[page])[:, :fill] * old[:, None, None]
                after = values(now[page])[:, :fill] * got[:, None, None]
                grown = got > was_scale[page].to(F)
                move = code_slip(before, got[:, None, None], codes) + 2.0 ** -20 * got[:, None, None] * QMAX[codes]
                assert torch.all((after - before).abs()[grown] <= move.expand_as(after)[grown])
                assert torch.equal(raw[page][~grown][:, :fill], raw_was[page][~grown][:, :fill])
            same[page, :j - lo] = False
            same_scale[page] = False
    keep = same[:, None, :, None].expand_as(raw)
    assert torch.equal(raw[keep], raw_was[keep])
    assert torch.equal(now_scale[same_scale], was_scale[same_scale])


BATCHES = {
    "first token": ([0], [1]),
    "one each": ([0, 5, 63, 64, 65, 127, 200, 31], [1] * 8),
    "some none": ([0, 7, 16, 100], [3, 0, 1, 0]),
    "fills a page": ([0, 16, 10, 48], [64, 48, 54, 16]),
    "prompts": ([0, 300, 17, 0, 63], [130, 65, 1, 257, 66]),
    "many pages": ([3], [1000]),
}


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D, page, H, Hq", [(64, 16, 3, 6), (128, 64, 2, 5), (256, 32, 1, 4), (128, 128, 1, 0), (64, 256, 2, 2)])
@pytest.mark.parametrize("name", BATCHES)
def test_append(d, name, D, page, H, Hq, dtype, codes, interleaved):
    print(f"append {name} D={D} page={page} H={H} Hq={Hq} {dtype} {codes} interleaved={interleaved}", flush=True)
    past, new = BATCHES[name]
    t, c = TYPES[dtype], CODES[codes]
    cache, table, cu, g = make(past, new, H, D, page, c, len(name) + D + page)
    T = cu[-1]
    qkv = torch.randn((T, Hq + 2 * H, D), generator=g, device=DEV)
    qkv *= torch.exp(torch.randn((T, Hq + 2 * H, 1), generator=g, device=DEV) * 0.5)
    qkv = qkv.to(t)
    q, k, v = (qkv[:, :Hq] if Hq else None), qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    rot = D if page != 32 else D // 4
    rope = decode.rope_table(table.shape[1] * page, rot)
    was = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    got_q = d.kv_append(cache, k, v, table.to(DEV), put(past), put(cu), max(new), q=q, rope=rope,
                        interleaved=interleaved)
    pos = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(past, new)])
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=F, device=DEV) / rot)
    check_store(cache, was[0], was[2], cache.k, cache.k_scale, rotate(k, pos, freq, interleaved), table, past, new, cu)
    check_store(cache, was[1], was[3], cache.v, cache.v_scale, v.to(F), table, past, new, cu)
    if Hq == 0:
        assert got_q is None
        return
    want = rotate(q, pos, freq, interleaved)
    # two products and a sum in binary32, with a table in binary32; then one rounding
    size = rotate(q.abs(), pos * 0, freq, interleaved).abs().amax(-1, keepdim=True) * 2
    tol = half_step(t) * want.abs() + 2.0 ** -22 * size + (torch.finfo(t).tiny * torch.finfo(t).eps)
    assert torch.all((got_q.to(F) - want).abs() <= tol)


@pytest.mark.parametrize("codes", CODES)
def test_exact_values_stay_exact(d, codes):
    """Powers of two and whole numbers that the codes hold come back as they went in."""
    c = CODES[codes]
    cache = decode.KvCache.empty(4, 1, 64, 16, c)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(-16, 17, (20, 1, 64), generator=g, device=DEV).half()
    x[:, :, 0] = QMAX[c]  # scale 1
    table = put([[2, 0, 3]])
    d.kv_append(cache, x, -x, table, put([0]), put([0, 20]), 20)
    assert torch.equal(cache.k_scale[[2, 0], 0], torch.ones(2, device=DEV))
    k, v = d.kv_read(cache, table, put([0]), put([0, 20]), tokens=20)
    assert torch.equal(k, x) and torch.equal(v, -x)


@pytest.mark.parametrize("codes", CODES)
def test_scale_grows_by_two_and_codes_halve(d, codes):
    c = CODES[codes]
    cache = decode.KvCache.empty(3, 2, 128, 16, c)
    table = put([[1, 2]])
    x = torch.zeros((3, 2, 128), device=DEV).bfloat16()
    x[:, :, 5] = QMAX[c]
    x[:, :, 7] = 6
    d.kv_append(cache, x, x, table, put([0]), put([0, 3]), 3)
    y = x[:1] * 2
    d.kv_append(cache, y, x[:1], table, put([3]))
    assert torch.all(cache.k_scale[1] == 2) and torch.all(cache.v_scale[1] == 1)
    k, v = d.kv_read(cache, table, put([0]), put([0, 4]), tokens=4, dtype=torch.bfloat16)
    # 224 is an e4m3 code, 63.5 rounds to the even 64 of the int8 ones
    assert torch.all(k[:3, :, 5] == (QMAX[c] if codes == "e4m3" else 128)) and torch.all(k[:3, :, 7] == 6)
    assert torch.equal(k[3], y[0]) and torch.equal(v[:3], x)


def test_first_slot_forgets_the_old_scale(d):
    cache = decode.KvCache.empty(2, 1, 64, 16)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(1e30)
    x = torch.ones((1, 1, 64), device=DEV).half()
    d.kv_append(cache, x, x, put([[1]]), put([0]))
    assert float(cache.k_scale[1, 0]) == pytest.approx(1 / 127, rel=1e-6)
    assert torch.isnan(cache.k_scale[0]).all() and float(cache.v_scale[1, 0]) == pytest.approx(1 / 127, rel=1e-6)


@pytest.mark.parametrize("codes", CODES)
def test_zeros_and_non_finite_values(d, codes):
    cache = decode.KvCache.empty(6, 1, 64, 16, CODES[codes])
    x = torch.zeros((3, 1, 64), device=DEV).half()
    x[1, 0, 3] = float("inf")
    x[2, 0, 9] = float("nan")
    table = put([[0], [2], [4]])
    d.kv_append(cache, x, torch.zeros_like(x), table, put([0, 0, 0]))
    k, v = d.kv_read(cache, table, put([0, 0, 0]))
    assert torch.all(k[0] == 0) and torch.all(v == 0)
    assert not torch.isfinite(k[1]).any() and torch.isnan(k[2]).all()
    d.kv_append(cache, torch.ones_like(x), torch.ones_like(x), table, put([1, 1, 1]))  # the damage stays visible
    k, v = d.kv_read(cache, table, put([1, 1, 1]))
    assert (k[0].float() - 1).abs().max() < 2 ** -9 and not torch.isfinite(k[1:]).any() and (v.float() - 1).abs().max() < 2 ** -9


def test_bad_pages_and_ends_are_skipped(d):
    """Entries that name no page, and positions past the table, take nothing and read as zeros."""
    cache = decode.KvCache.empty(4, 1, 64, 16)
    table = put([[-1, 1], [4, 2], [3, 0], [2 ** 31 - 1, -2 ** 31]])
    x = torch.ones((4 * 40, 1, 64), device=DEV).half()
    cu = put([0, 40, 80, 120, 160])
    rope = decode.rope_table(32, 64)
    q = d.kv_append(cache, x, x, table, put([0, 0, 0, 0]), cu, 40, q=x, rope=rope)
    assert torch.isfinite(q).all()
    k, v = d.kv_read(cache, table, put([0, 0, 0, 0]), cu, tokens=160)
    assert torch.all(cache.k_scale != 0)
    v = v.view(4, 40, 64)
    assert torch.all(v[:, 32:] == 0) and torch.all(v[0, :16] == 0) and torch.all(v[1, :16] == 0) and torch.all(v[3] == 0)
    assert torch.all(v[2, :32] != 0) and torch.all(v[0, 16:32] != 0) and torch.all(v[1, 16:32] != 0)
    k, v = d.kv_read(cache, table, put([-5, 40, 2 ** 31 - 1, 31]))
    assert torch.all(k == 0) and torch.all(v == 0)
    before = cache.k.clone()
    d.kv_append(cache, x[:4] * 2, x[:4], table, put([32, 2 ** 31 - 1, 33, 40]))
    assert torch.equal(before, cache.k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("D, page, H", [(64, 16, 5), (128, 64, 8), (256, 128, 1)])
def test_read(d, D, page, H, codes, dtype):
    past, new = [0, 10, 130, 64], [70, 0, 5, 64]
    cache, table, cu, g = make(past, new, H, D, page, CODES[codes], 4)
    t = TYPES[dtype]
    k, v = d.kv_read(cache, table.to(DEV), put(past), put(cu), tokens=cu[-1], max_tokens=70, dtype=t)
    for got, buf, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        for b in range(4):
            for i in range(new[b]):
                p = past[b] + i
                page_id = int(table[b, p // page])
                want = values(buf[page_id, :, p % page]) * scale[page_id].to(F)[:, None]
                err = (got[cu[b] + i].to(F) - want).abs()
                assert torch.all(err <= (half_step(t) * (1 + 2.0 ** -10) + 2.0 ** -24) * want.abs() + (torch.finfo(t).tiny * torch.finfo(t).eps))


def test_in_place_queries_and_a_graph(d):
    """q turned in place inside a fused projection; captured and replayed between eager work."""
    H, Hq, D, page, B = 2, 4, 128, 32, 3
    cache, table, cu, g = make([40, 0, 31], [1, 1, 1], H, D, page, torch.int8, 8)
    table, rope = table.to(DEV), decode.rope_table(64 * 2, D)
    past = put([40, 0, 31])
    qkv = torch.randn((B, Hq + 2 * H, D), generator=g, device=DEV).half()
    src = qkv.clone()
    start = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    want_q = d.kv_append(cache, src[:, Hq:Hq + H], src[:, Hq + H:], table, past, q=src[:, :Hq], rope=rope)
    want = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        d.kv_append(cache, qkv[:, Hq:Hq + H], qkv[:, Hq + H:], table, past, q=qkv[:, :Hq], rope=rope, q_out=qkv[:, :Hq])
    for _ in range(3):
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), start):
            x.copy_(y)
        qkv.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qkv[:, :Hq], want_q) and torch.equal(qkv[:, Hq:], src[:, Hq:])
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_offsets_past_32_bits(d):
    """A cache of over 4 GiB a side: the last pages are written and read."""
    pages = 2 ** 32 // (8 * 256 * 256) + 40
    shape = (pages, 8, 256, 256)
    cache = decode.KvCache(torch.empty(shape, dtype=torch.int8, device=DEV), torch.empty(shape, dtype=torch.int8, device=DEV),
                           *[torch.zeros((pages, 8), device=DEV) for _ in range(2)])
    assert cache.k.numel() > 2 ** 32
    x = torch.randn((300, 8, 256), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).half()
    table = put([[pages - 1, pages - 2]])
    d.kv_append(cache, x, -x, table, put([0]), put([0, 300]), 300)
    k, v = d.kv_read(cache, table, put([0]), put([0, 300]), tokens=300)
    step = x.float().abs().max() / 127
    assert (k.float() - x.float()).abs().max() <= step * 0.51 and (v.float() + x.float()).abs().max() <= step * 0.51


def test_refusals_on_the_device(d):
    cache = decode.KvCache.empty(4, 2, 64, 16)
    x = torch.zeros((1, 2, 64), device=DEV).half()
    table, past = put([[0, 1]]), put([0])
    good = dict(cache=cache, k=x, v=x, table=table, past=past, q=x, rope=decode.rope_table(32, 64))
    d.kv_append(**good)
    for bad in (dict(k=x[:, :1]), dict(v=x.bfloat16()), dict(k=x.float(), v=x.float()), dict(table=table.long()),
                dict(past=past.long()), dict(past=put([0, 0])), dict(table=table[0]), dict(rope=decode.rope_table(31, 64)),
                dict(rope=decode.rope_table(32, 64).half()), dict(q=x[..., :32]), dict(table=table.cpu()),
                dict(cu_new=put([0, 1, 1])), dict(q_out=torch.zeros((2, 2, 64), device=DEV).half())):
        with pytest.raises((ValueError, TypeError)):
            d.kv_append(**{**good, **bad})
    with pytest.raises(decode.DecodeError):
        d.kv_append(**{**good, "rope": decode.rope_table(32, 24)})
    with pytest.raises(TypeError):
        d.kv_read(cache, table, past, dtype=torch.float32)
    for args in ((cache.k, cache.v[:, :1], cache.k_scale, cache.v_scale), (cache.k.float(), cache.v.float(), cache.k_scale, cache.v_scale),
                 (cache.k, cache.v, cache.k_scale[:2], cache.v_scale), (cache.k, cache.v, cache.k_scale.half(), cache.v_scale),
                 (cache.k.transpose(1, 2), cache.v.transpose(1, 2), cache.k_scale, cache.v_scale)):
        with pytest.raises((ValueError, TypeError)):
            decode.KvCache(*args)
