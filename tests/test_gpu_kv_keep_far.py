"""kv_keep between pages that lie past 4 GiB."""
import pytest
import torch

from decode_ref import F

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)


def put(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("to_far", [False, True])
@pytest.mark.parametrize("kept", [[10], list(range(10, 260))])
def test_codes_and_scales(to_far, kept):
    """One token, which comes from another page, and a path that is longer than a workgroup holds."""
    H, D, ps, past = 8, 128, 256, 250
    pages = (5 << 30) // (H * ps * D)
    cache = decode.KvCache.empty(pages, H, D, ps)
    near, far = [2, 5], [pages - 2, pages - 7]
    table = [near[0], far[0], near[1]] if not to_far else [far[0], near[0], far[1]]
    gen = torch.Generator(device="cuda").manual_seed(len(kept))
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        for i, page in enumerate(table):
            x[page] = torch.randint(-127, 128, (H, ps, D), device="cuda", generator=gen, dtype=torch.int8)
            s[page] = 2.0 ** (i - 3)  # each page's values are larger than the ones before
    untouched = [p for p in (0, 1, 3, pages - 1, pages - 3, (pages - 2) - (1 << 32) // (H * ps * D)) if p not in table]
    was = [(x[table].clone(), s[table].clone()) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    with decode.Decode() as d:
        d.kv_keep(cache, put([table]), put([past]), put(kept), put([0, len(kept)]))
    for (old, scale), x, s in zip(was, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        value = old.to(F) * scale.to(F)[..., None, None]
        value, page_of = value.transpose(1, 2).reshape(3 * ps, H, D), torch.arange(3 * ps) // ps
        for page in range(3):
            places = [p for p in range(past, past + len(kept)) if p // ps == page]
            come = [past + kept[p - past] for p in places]
            other = [c for c in come if page_of[c] != page]
            want = scale[page].to(F)
            if other:
                want = torch.maximum(want, value[other].abs().amax((0, 2)) / 127)
            # the largest value and its quotient are two roundings
            assert torch.all((s[table[page]].to(F) - want).abs() <= want * 2.0 ** -22)
            grows = bool((want > scale[page].to(F)).any())
            got = x[table[page]].to(F).transpose(0, 1)  # [slot, head, channel]
            held = list(range(past % ps)) if page == past // ps else []
            for slots, rows in (([p % ps for p in places], value[come] if come else None), (held, value[[page * ps + p for p in held]] if held else None)):
                if rows is None:
                    continue
                exact = rows / want[:, None]
                # a code is within half of the quotient, and scale, ratio and product are five roundings
                assert torch.all((got[slots] - exact).abs() <= 0.5 * (1 + 2.0 ** -20) + 127 * 5 * 2.0 ** -24)
            rest = [i for i in range(ps) if i not in held and page * ps + i not in places]
            assert torch.equal(x[table[page]][:, rest], old[page][:, rest])
            assert grows == bool(other)
        assert not x[untouched].any() and not s[untouched].any()
