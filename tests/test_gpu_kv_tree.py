"""kv_attend_tree on the GPU against attention over each row's own tokens in float64."""
import math
import random

import pytest
import torch

from decode_ref import layout, random_codes
from drafts_ref import attend_tree, check_attend

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda", 0)
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


def put(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def trees(new, seed, words=None):
    """Bits of a random tree for each sequence, rows one after the other."""
    r = random.Random(seed)
    words = -(-max(new + [1]) // 32) if words is None else words
    out = torch.zeros((sum(new), words), dtype=torch.int32)
    at = 0
    for n in new:
        bits, _ = decode.tree([r.randint(max(-1, i - 5), i - 1) for i in range(n)])
        out[at:at + n, :bits.shape[1]] = bits
        at += n
    return out.to(DEV)


def make(lens, new, Hq, Hkv, D, page, code, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    dgen = torch.Generator(device=DEV).manual_seed(seed)
    pages = sum(-(-max(n, 0) // page) for n in lens) + 2
    k, v = (random_codes((pages, Hkv, page, D), code, dgen) for _ in range(2))
    ks, vs = (torch.exp(torch.randn((pages, Hkv), device=DEV, generator=dgen) * 0.3) / 60 for _ in range(2))
    cache = decode.KvCache(k, v, ks, vs)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], Hq, D), device=DEV, generator=dgen).to(dtype)
    return cache, layout(lens, page, pages, gen, extra_cols=1), cu, q


def run(d, lens, new, Hq, Hkv, D, page, code=torch.int8, dtype=torch.float16, seed=0, bits=None, **kw):
    cache, table, cu, q = make(lens, new, Hq, Hkv, D, page, code, dtype, seed)
    bits = trees(new, seed) if bits is None else bits
    got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), max(new), max_len=max(lens), **kw)
    check_attend(got, *attend_tree(q, cache, table, lens, bits, cu, **kw))
    return cache, table, cu, q, bits, got


@pytest.mark.parametrize("code", [torch.int8, E4M3])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G, new", [(1, [5, 1, 12]), (4, [12, 3, 7]), (8, [8, 1, 4]), (8, [33, 7, 1]), (5, [64, 30, 2]), (4, [130, 65, 5])])
def test_against_the_definition(d, code, dtype, D, G, new):
    """From one 16-row tile to several blocks of the kernel for many rows."""
    lens = [n + c for n, c in zip(new, (300, 0, 77))]
    run(d, lens, new, 2 * G, 2, D, 32, code, dtype, seed=D + G)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n, context", [(1, 0), (1, 31), (2, 30), (12, 16), (31, 1), (32, 32), (33, 63), (64, 64), (65, 127), (40, 129)])
def test_drafts_at_every_place(d, page, n, context):
    """Drafts that begin and end inside tiles, words and pages."""
    for D, G in ((128, 2), (64, 8)):
        run(d, [context + n], [n], 2 * G, 2, D, page, seed=n + context)


@pytest.mark.parametrize("window, sinks", [(1, 0), (5, 2), (40, 0), (64, 70), (1000, 4), (10 ** 9, 0)])
@pytest.mark.parametrize("code", [torch.int8, E4M3])
def test_windows(d, window, sinks, code):
    for new, G, D in (([9, 1, 14], 4, 128), ([70, 33, 2], 4, 64), ([20, 5, 9], 8, 256)):
        lens = [n + c for n, c in zip(new, (700, 3, 130))]
        run(d, lens, new, 2 * G, 2, D, 16, code, seed=window % 97, window=window, sinks=sinks)


def test_split_contexts(d):
    """Long contexts of few sequences: blocks in parts, joined by the last workgroup or a second kernel."""
    for new, G, context, H in (([12], 4, 4096, 8), ([3], 1, 9000, 1), ([48], 4, 20000, 2), ([64, 64], 8, 7000, 1), ([130], 8, 9000, 1)):
        run(d, [context + n for n in new], new, G * H, H, 128, 64, torch.int8, torch.bfloat16, seed=context)


def test_a_chain_is_attention_in_order(d):
    """Every token sees those before it: kv_attend's result up to both kernels' roundings."""
    for new in ([6, 1, 20], [100, 64, 3]):
        lens = [n + c for n, c in zip(new, (500, 40, 0))]
        bits = torch.cat([decode.tree(range(-1, n - 1))[0] if n > max(new) - 32 else
                          torch.nn.functional.pad(decode.tree(range(-1, n - 1))[0], (0, -(-max(new) // 32) - -(-n // 32)))
                          for n in new]).to(DEV)
        cache, table, cu, q, _, got = run(d, lens, new, 8, 2, 128, 32, bits=bits, seed=3)
        same = d.kv_attend(q, cache, table.to(DEV), put(lens), put(cu), max(new))
        # the walks over tiles are not the same (a tree's rows all go on to the last token), so neither are the sums'
        # orders: each is within the bound of the exact result
        check_attend(same, *attend_tree(q, cache, table, lens, bits, cu))
        got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), max(new), window=50, sinks=3)
        ref, bound = attend_tree(q, cache, table, lens, bits, cu, 50, 3)
        check_attend(got, ref, bound)


def test_masks_that_are_no_tree(d):
    """Any bits: tokens that see later ones, none but themselves, all, or none at all; bits past the drafts say nothing."""
    new, lens = [10, 40, 3], [10, 47, 503]
    gen = torch.Generator(device=DEV).manual_seed(5)
    bits = torch.randint(-2 ** 31, 2 ** 31, (53, 2), device=DEV, generator=gen, dtype=torch.int64).int()
    bits[0], bits[11], bits[52] = 0, 0, 0
    bits[1] = -1
    for G in (1, 8):
        cache, table, cu, q, _, got = run(d, lens, new, 2 * G, 2, 64, 16, bits=bits, seed=8)
        assert torch.all(got[0] == 0)  # no context, and no bit
        run(d, lens, new, 2 * G, 2, 64, 16, bits=bits, seed=9, window=8, sinks=1)


def test_more_words_than_are_needed_and_rows_apart(d):
    new, lens = [5, 33], [105, 33]
    wide = trees(new, 4, words=7)
    _, _, _, _, _, a = run(d, lens, new, 8, 2, 128, 32, bits=wide, seed=2)
    _, _, _, _, _, b = run(d, lens, new, 8, 2, 128, 32, bits=wide[:, :2], seed=2)
    assert torch.equal(a, b) and wide[:, :2].stride(0) == 7


@pytest.mark.parametrize("new", [[7, 3], [60, 20]])
def test_hidden_nan_codes_do_not_matter_and_seen_ones_do(d, new):
    lens = [n + 50 for n in new]
    cache, table, cu, q = make(lens, new, 16, 2, 128, 16, E4M3, torch.float16, 11)
    bits = trees(new, 12)
    want = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), max(new))
    # the first sequence's third draft; behind its end; and a page of no sequence
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    at = 52
    for x in (k, v):
        x[table[0, at // 16].item(), :, at % 16, 5] = 0x7f
        end = lens[0]
        if end % 16:
            x[table[0, end // 16].item(), :, end % 16:] = 0x7f
    got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), max(new))
    sees = (bits[:new[0], 0] >> 2 & 1).bool()
    assert sees.any() and not sees.all()
    assert torch.isnan(got[:new[0]][sees]).any(-1).all()
    assert torch.equal(got[:new[0]][~sees], want[:new[0]][~sees])
    assert torch.equal(got[new[0]:], want[new[0]:])


def test_pages_that_are_not_there(d):
    """A page number outside the cache hides its tokens, context or drafts."""
    new, lens = [20, 6], [100, 70]
    for G in (1, 8):
        cache, table, cu, q = make(lens, new, 2 * G, 2, 64, 16, torch.int8, torch.float16, 21)
        bits = trees(new, 22)
        table[0, 2], table[0, 5], table[1, 4] = -1, 1 << 30, cache.pages
        got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), max(new))
        check_attend(got, *attend_tree(q, cache, table, lens, bits, cu))


def test_rows_of_no_sequence_stay(d):
    """Tokens before cu[0] and from cu[batch] on are not written; sequences without drafts have no rows."""
    lens, cu = [50, 60, 31], [2, 9, 9, 13]
    for Hq in (4, 32):
        cache, table, _, _ = make(lens, [7, 0, 4], Hq, 2, 128, 32, torch.int8, torch.float16, 31)
        q = torch.randn((17, Hq, 128), device=DEV).half()
        bits = torch.zeros((17, 1), dtype=torch.int32, device=DEV)
        bits[2:9], bits[9:13] = decode.tree([-1, 0, 0, 1, 1, 2, 2])[0].to(DEV), decode.tree([-1, -1, 0, 1])[0].to(DEV)
        out = torch.full_like(q, 7)
        d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), 7, out=out)
        assert torch.all(out[:2] == 7) and torch.all(out[13:] == 7)
        ref, bound = attend_tree(q, cache, table, lens, bits, cu)
        check_attend(out[2:13], ref[2:13], bound[2:13])


def test_lengths_that_do_not_fit(d):
    """Fewer tokens than drafts, none, negative ones, and more than the table has: nothing out of place is read."""
    new = [10, 5, 4, 6]
    cache, table, cu, q = make([40, 40, 40, 64], new, 8, 2, 64, 16, torch.int8, torch.float16, 41)
    bits = trees(new, 42)
    lens = [6, 0, -3, 10 ** 9]
    got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), 10)
    assert torch.all(got[cu[1]:cu[3]] == 0)
    check_attend(got, *attend_tree(q, cache, table, lens, bits, cu))


def test_one_token_without_cu(d):
    lens = [5, 300, 77]
    cache, table, cu, q = make(lens, [1, 1, 1], 8, 2, 128, 32, E4M3, torch.bfloat16, 51)
    bits = put([[1], [1], [0]])
    got = d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits)
    check_attend(got, *attend_tree(q, cache, table, lens, bits, cu))


def test_many_sequences(d):
    """More row blocks than one lane each: the walk along the line of work goes on."""
    r = random.Random(1)
    new = [r.randint(0, 9) for _ in range(150)]
    lens = [n + r.randint(0, 90) for n in new]
    run(d, lens, new, 8, 2, 64, 16, seed=61)


def test_in_a_graph_with_other_lengths_and_trees(d):
    new, cap = [9, 4], 400
    cache, table, cu, q = make([cap, cap], new, 16, 2, 128, 32, torch.int8, torch.float16, 71)
    dt, lens, bits = table.to(DEV), put([100, 80]), trees(new, 72)
    call = lambda: d.kv_attend_tree(q, cache, dt, lens, bits, put_cu, 9, max_len=cap)  # noqa: E731
    put_cu = put(cu)
    call()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = call()
    for seed, now in ((1, [9, 4]), (2, [400, 250]), (3, [33, 390])):
        lens.copy_(put(now))
        bits.copy_(trees(new, seed))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())
        check_attend(out, *attend_tree(q, cache, table, now, bits, cu))


def test_the_same_bits_every_time(d):
    cache, table, cu, q = make([9000, 500], [20, 12], 32, 8, 128, 64, torch.int8, torch.float16, 81)
    bits, args = trees([20, 12], 82), (put([9000, 500]),)
    want = d.kv_attend_tree(q, cache, table.to(DEV), *args, bits, put(cu), 20)
    for _ in range(5):
        assert torch.equal(d.kv_attend_tree(q, cache, table.to(DEV), *args, bits, put(cu), 20), want)


def test_refusals(d):
    lens, new = [50, 60], [40, 5]
    cache, table, cu, q = make(lens, new, 8, 2, 64, 16, torch.int8, torch.float16, 91)
    bits = trees(new, 92)
    call = lambda bits, **kw: d.kv_attend_tree(q, cache, table.to(DEV), put(lens), bits, put(cu), **{"max_q": 40, **kw})  # noqa: E731
    with pytest.raises(TypeError):
        call(bits.long())
    with pytest.raises(TypeError):
        call(None)
    for bad in (bits[:, :1], bits[:44], bits[0], bits.t().contiguous().t(), bits.cpu()):
        with pytest.raises(ValueError):
            call(bad)
    with pytest.raises(ValueError):
        call(bits, window=-1)
    with pytest.raises(decode.DecodeError):
        call(bits, scale=math.inf)


@pytest.mark.parametrize("D, Hkv, new", [(128, 8, 64), (64, 2, 64), (256, 2, 130)])
def test_very_uneven_lengths(d, D, Hkv, new):
    """Many rows, one long sequence among short, empty and middling ones: parts by length, some joined and some not."""
    r = random.Random(D)
    n = [r.randint(1, new) for _ in range(12)]
    n[0], n[5], n[7] = new, 0, new
    lens = [a + c for a, c in zip(n, [20000, 3, 0, 700, 64, 100, 2000, 10000, 1, 63, 5000, 257])]
    run(d, lens, n, 4 * Hkv, Hkv, D, 64, torch.int8, torch.float16, seed=D, window=0)
    run(d, lens, n, 4 * Hkv, Hkv, D, 64, E4M3, torch.bfloat16, seed=D, window=3000, sinks=100)


def test_more_row_blocks_than_lanes_with_many_rows(d):
    """Over 64 row blocks on the line, most of them short."""
    r = random.Random(2)
    n = [r.randint(0, 40) for _ in range(100)]
    n[3] = n[80] = 40
    lens = [a + r.choice((0, 5, 200, 900)) for a in n]
    lens[3], lens[80] = 6000, 9000
    run(d, lens, n, 8, 2, 64, 16, seed=62)
