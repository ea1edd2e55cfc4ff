"""kv_keep and kv_copy on the GPU: moves of tokens and pages against their definitions."""
import math
import random

import pytest
import torch

from decode_ref import F, QMAX, half_step, layout, random_codes, values
from drafts_ref import STEP32, keep

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda", 0)
E4M3 = torch.float8_e4m3fn
PARTS = (("k", "k_scale"), ("v", "v_scale"))


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


def put(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def new_cache(pages, H, page, D, code, seed, spread=0.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    k, v = (random_codes((pages, H, page, D), code, gen) for _ in range(2))
    ks, vs = (torch.exp(torch.randn((pages, H), device=DEV, generator=gen) * spread) / 60 for _ in range(2))
    return decode.KvCache(k, v, ks, vs)


def clone(cache):
    return decode.KvCache(*[getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")])


def same(x, y):
    return torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def check_keep(before, after, table, past, kept, cu):
    most = QMAX[before.k.dtype]
    for part, name in PARTS:
        rows, scale = keep(getattr(before, part), getattr(before, name), table, past, kept, cu)
        got = getattr(after, name).to(F)
        # the largest value and its quotient are two roundings
        assert torch.all((got - scale).abs() <= scale.abs() * 2 * STEP32 * 1.01)
        was, now = getattr(before, part).view(torch.uint8), getattr(after, part).view(torch.uint8)
        touched = torch.zeros(was.shape[:3], dtype=torch.bool, device=DEV)
        for page, slot, want, exact in rows:
            touched[page, :, slot] = True
            have = values(getattr(after, part)[page, :, slot])
            want = want.clamp(-most, most)
            # scale, ratio and product are five roundings before the code's own
            slip = want.abs() * 5 * STEP32 * 1.01
            near = 0.5 if before.k.dtype == torch.int8 else torch.maximum(half_step(E4M3) * want.abs(), torch.full_like(want, 2.0 ** -10))
            assert torch.all((have - want).abs() <= near * (1 + 2.0 ** -20) + slip), (part, page, slot)
            assert torch.equal(have[exact], want[exact])
        assert torch.equal(now[~touched], was[~touched])


def case(past, drafts, path, page, H=2, D=64, code=torch.int8, seed=0, extra=0):
    lens = [p + n for p, n in zip(past, drafts)]
    pages = sum(-(-n // page) for n in lens) + 3
    table = layout(lens, page, pages, torch.Generator().manual_seed(seed), extra_cols=extra)
    cu = [0]
    for p in path:
        cu.append(cu[-1] + len(p))
    return new_cache(pages, H, page, D, code, seed), table, sum(path, []), cu


def run(d, past, drafts, path, page, **kw):
    cache, table, kept, cu = case(past, drafts, path, page, **kw)
    before = clone(cache)
    d.kv_keep(cache, table.to(DEV), put(past), put(kept), put(cu), max([len(p) for p in path] + [1]))
    check_keep(before, cache, table.tolist() and table, past, kept, cu)
    return before, cache, table


@pytest.mark.parametrize("code", [torch.int8, E4M3])
@pytest.mark.parametrize("page, D, H", [(16, 64, 2), (32, 128, 3), (64, 256, 1), (128, 128, 2), (256, 64, 1)])
def test_paths(d, code, page, D, H):
    """Paths that stay on a page, cross pages, skip whole pages, and keep all."""
    r = random.Random(page)
    past = [0, 5, page - 1, page, 3 * page + 7]
    drafts = [12, 40, 3 * page + 3, 70, 64]
    path = [sorted(r.sample(range(n), r.randint(1, n))) for n in drafts]
    path[3] = list(range(70))
    path[4] = list(range(0, 64, 7))
    run(d, past, drafts, path, page, code=code, D=D, H=H, seed=page + D)


@pytest.mark.parametrize("code", [torch.int8, E4M3])
def test_long_paths(d, code):
    """More tokens than a workgroup moves at a time, over many pages."""
    r = random.Random(4)
    for D, page in ((256, 64), (64, 32), (128, 256)):
        path = [sorted(r.sample(range(700), 400)), list(range(1, 600)), sorted(r.sample(range(650), 3))]
        run(d, [11, 100, 0], [700, 600, 650], path, page, code=code, D=D, seed=D)


def test_indices_that_do_not_ascend(d):
    """The same token more than once, later ones before earlier ones, and entries that say nothing."""
    path = [[3, 3, 9, 3, 9], [5, 4, 3, 2, 1], [2, 0, -1, 3, 2 ** 31 - 1], [-5], [0, 1, 2]]
    run(d, [10, 14, 30, 3, 0], [12, 20, 12, 4, 3], path, 16, seed=3)


def test_nothing_moves(d):
    """All drafts kept, or none: every byte stays."""
    for path in ([list(range(12)), list(range(30))], [[], []], [[], list(range(5))]):
        before, after, _ = run(d, [10, 40], [12, 30], path, 16, seed=5)
        for n in ("k", "v", "k_scale", "v_scale"):
            assert same(getattr(before, n), getattr(after, n))


def test_one_each_without_cu(d):
    past, kept = [7, 31, 0], [4, 9, 0]
    cache, table, _, _ = case(past, [10, 10, 10], [[4], [9], [0]], 16, seed=6)
    before = clone(cache)
    d.kv_keep(cache, table.to(DEV), put(past), put(kept))
    check_keep(before, cache, table, past, kept, [0, 1, 2, 3])


def test_pages_that_are_not_there(d):
    """A position without a page is skipped, one whose source has none stays."""
    path = [list(range(2, 60, 2)), list(range(1, 40))]
    cache, table, kept, cu = case([10, 3], [60, 40], path, 16, seed=7)
    table[0, 1], table[0, 3], table[1, 2] = -1, 1 << 20, cache.pages
    before = clone(cache)
    d.kv_keep(cache, table.to(DEV), put([10, 3]), put(kept), put(cu))
    check_keep(before, cache, table, [10, 3], kept, cu)


def test_lengths_that_do_not_fit(d):
    """Negative lengths count as none, and positions past the table as no page."""
    path = [[1, 3], [0, 5, 7, 30], [2]]
    cache, table, kept, cu = case([0, 60, 40], [12, 4, 8], path, 16, seed=8)
    past = [-4, 60, 10 ** 9]
    before = clone(cache)
    d.kv_keep(cache, table.to(DEV), put(past), put(kept), put(cu))
    check_keep(before, cache, table, past, kept, cu)


def test_scales_of_zero_and_of_very_different_sizes(d):
    for code in (torch.int8, E4M3):
        path = [list(range(3, 60, 3)), list(range(20, 50))]
        cache, table, kept, cu = case([20, 9], [60, 50], path, 16, code=code, seed=9)
        for s in (cache.k_scale, cache.v_scale):
            s.copy_(torch.exp2(torch.randint(-40, 41, s.shape, device=DEV).float()))
            s[table[0, 2].item()] = 0
            s[table[1, 1].item()] = 0
            s[table[1, 3].item(), 0] = 0
        before = clone(cache)
        d.kv_keep(cache, table.to(DEV), put([20, 9]), put(kept), put(cu))
        check_keep(before, cache, table, [20, 9], kept, cu)


def test_scales_that_are_not_finite(d):
    """They reach the pages that tokens from theirs come to, in their head, and no other."""
    path = [[20, 21], [1, 2]]
    cache, table, kept, cu = case([4, 4], [40, 8], path, 16, seed=10)
    want = clone(cache)
    d.kv_keep(want, table.to(DEV), put([4, 4]), put(kept), put(cu))
    for bad in (math.inf, math.nan):
        c, _, _, _ = case([4, 4], [40, 8], path, 16, seed=10)
        c.k_scale[table[0, 1].item(), 1] = bad  # positions 24 and 25
        d.kv_keep(c, table.to(DEV), put([4, 4]), put(kept), put(cu))
        assert not torch.isfinite(c.k_scale[table[0, 0].item(), 1])
        c.k_scale[table[0, 0].item(), 1] = want.k_scale[table[0, 0].item(), 1]
        c.k_scale[table[0, 1].item(), 1] = want.k_scale[table[0, 1].item(), 1]
        c.k[table[0, 0].item(), 1] = want.k[table[0, 0].item(), 1]
        for n in ("k", "v", "k_scale", "v_scale"):
            assert same(getattr(c, n), getattr(want, n)), n


def test_tokens_of_no_sequence_and_empty_calls(d):
    """Entries before cu[0] and from cu[batch] on belong to nobody."""
    past, drafts = [10, 20], [20, 20]
    cache, table, _, _ = case(past, drafts, [[1], [1]], 16, seed=11)
    before = clone(cache)
    kept, cu = [9, 9, 2, 5, 3, 7, 9], [2, 4, 6]
    d.kv_keep(cache, table.to(DEV), put(past), put(kept), put(cu))
    check_keep(before, cache, table, past, kept, cu)
    d.kv_keep(cache, table[:0].to(DEV), put([]), put([]), put([0]))


def test_the_order_of_a_graphs_work(d):
    """Append, keep and read of one cache as nodes of a graph, replayed over fresh drafts."""
    page, H, D = 16, 2, 64
    cache = decode.KvCache.empty(12, H, D, page)
    table, past, cu = put([[3, 0, 7], [5, 2, 9]]), put([9, 20]), put([0, 10, 16])
    k, v = (torch.randn((16, H, D), device=DEV).half() for _ in range(2))
    kept, cuk = put([0, 3, 8, 1, 5]), put([0, 3, 5])

    def step():
        d.kv_append(cache, k, v, table, past, cu, 10)
        d.kv_keep(cache, table, past, kept, cuk, 3)
        return d.kv_read(cache, table, past, cuk, tokens=5, max_tokens=3)

    step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = step()
    rows = [0, 3, 8, 11, 15]
    for seed in range(3):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        for x in (k, v):
            x.copy_(torch.randn(x.shape, device=DEV, generator=gen).half())
        g.replay()
        torch.cuda.synchronize()
        for got, x, name in ((out[0], k, "k_scale"), (out[1], v, "v_scale")):
            # a code is within half a step when it is appended and again when its scale grows, and fp16 rounds it
            step_size = getattr(cache, name).max()
            assert torch.all((got.float() - x[rows].float()).abs() <= step_size * 1.01 + x[rows].float().abs() * 2.0 ** -10)


@pytest.mark.parametrize("code", [torch.int8, E4M3])
@pytest.mark.parametrize("pages, pairs, H, page, D", [(3, 1, 1, 16, 64), (40, 13, 3, 16, 64), (30, 9, 8, 64, 128), (25, 7, 5, 256, 256),
                                                     (600, 290, 2, 32, 128)])
def test_copies(d, code, pages, pairs, H, page, D):
    cache = new_cache(pages, H, page, D, code, pages)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
    src, dst = order[:pairs].clone(), order[pairs:2 * pairs]
    src[pairs // 2:] = src[0]  # one page several times
    want = clone(cache)
    for part, scale in PARTS:
        raw = getattr(want, part).view(torch.uint8)
        raw[dst.to(DEV)] = raw[src.to(DEV)]
        getattr(want, scale)[dst.to(DEV)] = getattr(want, scale)[src.to(DEV)]
    d.kv_copy(cache, src.int().to(DEV), dst.int().to(DEV))
    for n in ("k", "v", "k_scale", "v_scale"):
        assert same(getattr(cache, n), getattr(want, n)), n


def test_pairs_that_say_nothing(d):
    cache = new_cache(10, 2, 16, 64, torch.int8, 2)
    want = clone(cache)
    d.kv_copy(cache, put([-1, 3, 10, 4, 2 ** 31 - 1, 5]), put([1, -1, 2, 10, 6, 5]))
    d.kv_copy(cache, put([]), put([]))
    for n in ("k", "v", "k_scale", "v_scale"):
        assert same(getattr(cache, n), getattr(want, n)), n


def test_copies_past_4_gib(d):
    cache = new_cache(1, 8, 256, 128, torch.int8, 3)
    pages = (5 << 30) // (8 * 256 * 128)
    big = decode.KvCache.empty(pages, 8, 128, 256)
    big.k[3], big.v[3], big.k_scale[3], big.v_scale[3] = cache.k[0], cache.v[0], cache.k_scale[0], cache.v_scale[0]
    d.kv_copy(big, put([3]), put([pages - 1]))
    d.kv_copy(big, put([pages - 1]), put([1]))
    for part, scale in PARTS:
        for at in (pages - 1, 1):
            assert same(getattr(big, part)[at], getattr(cache, part)[0]) and same(getattr(big, scale)[at], getattr(cache, scale)[0])
    table, past = put([[2, pages - 2]]), put([250])
    big.k[pages - 2, :, 4], big.k_scale[pages - 2] = cache.k[0, :, 4], 1.0
    d.kv_keep(big, table, past, put([10]))
    assert same(big.k[2, :, 250], cache.k[0, :, 4]) or torch.all((big.k[2, :, 250].int() - cache.k[0, :, 4].int()).abs() <= 127)
    top = cache.k[0, :, 4].abs().amax(1).float() / 127
    assert torch.all((big.k_scale[2] - top).abs() <= top * 2.0 ** -22)


def test_refusals(d):
    cache = new_cache(10, 2, 16, 64, torch.int8, 4)
    one = put([1, 2])
    for bad in ((one.long(), one), (one, one.float())):
        with pytest.raises(TypeError):
            d.kv_copy(cache, *bad)
    for bad in ((one, put([1])), (one.cpu(), one), (one, put([[1, 2]])), (put([[1, 5], [2, 6]])[:, 0], one)):
        with pytest.raises(ValueError):
            d.kv_copy(cache, *bad)
    table, past = put([[1, 2], [3, 4]]), put([5, 6])
    with pytest.raises(TypeError):
        d.kv_keep(cache, table, past, one.long())
    for bad in ((table, past, put([1, 2, 3])), (table[:1], past, one), (table, past, one, put([0, 1])), (table, past.cpu(), one)):
        with pytest.raises(ValueError):
            d.kv_keep(cache, *bad)
    with pytest.raises(decode.DecodeError):
        d.kv_keep(cache, table, past, one, put([0, 1, 2]), 0)
