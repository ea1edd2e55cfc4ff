"""kv_keep on a page that holds a NaN code and whose scale grows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_kv_move import clone, new_cache, put  # noqa: E402


@pytest.mark.parametrize("kept", [[0, 5, 20, 21], [0, 5, *range(20, 160)]])
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_a_nan_on_a_page_stays_one(kept, code):
    """Of an earlier token, of one that keeps its place and of one that moves on its page; nothing else changes for it."""
    D, past = 64, 4
    cache = new_cache(12, 2, 16, D, torch.float8_e4m3fn, 5)
    cache.k_scale[1], cache.v_scale[1] = 1.0, 1.0  # where tokens 20 and 21 come from; page 0's scales grow by it
    want, table = clone(cache), put([list(range(12))])
    nans = [(2, 0), (past, 63), (past + 5, 17)]  # position and channel, all on page 0
    for x in (cache.k, cache.v):
        for pos, d in nans:
            x.view(torch.uint8)[0, :, pos, d] = code
    with decode.Decode() as d:
        for c in (cache, want):
            old = c.k_scale[0].clone()
            d.kv_keep(c, table, put([past]), put(kept), put([0, len(kept)]))
            assert torch.all(c.k_scale[0] > old)
    for name in ("k", "v"):
        got, ref = getattr(cache, name).view(torch.uint8), getattr(want, name).view(torch.uint8).clone()
        for pos, d in ((2, 0), (past, 63), (past + 1, 17)):
            assert torch.isnan(getattr(cache, name)[0, :, pos, d].float()).all()
            ref[0, :, pos, d] = got[0, :, pos, d]
        for pos, d in nans[2:]:  # the place that the moved token came from, which a later one of the path may take
            if torch.isnan(getattr(cache, name)[0, :, pos, d].float()).any():
                ref[0, :, pos, d] = got[0, :, pos, d]
        assert torch.equal(got, ref)
        assert torch.equal(getattr(cache, name + "_scale"), getattr(want, name + "_scale"))
