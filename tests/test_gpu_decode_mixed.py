"""Batches that mix a piece of a prompt with single tokens, as a server sends them, over short and long contexts."""
import pytest
import torch

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_decode_attend import CODES, DEV, check, make, put  # noqa: E402


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("window, sinks", [(0, 0), (700, 4)])
@pytest.mark.parametrize("D, Hq, H, batch", [(128, 8, 2, 5), (64, 4, 1, 70), (256, 16, 2, 4)])
def test_prompt_piece_and_single_tokens(d, D, Hq, H, batch, window, sinks, codes):
    new = [300] + [1] * (batch - 2) + [0]
    past = [1000, 30000, 0] + [17 * i % 500 for i in range(batch - 3)]
    lens = [p + n for p, n in zip(past, new)]
    cache, table, cu, q = make(lens, new, Hq, H, D, 64, CODES[codes], torch.bfloat16, D + batch)
    kw = dict(window=window, sinks=sinks)
    mixed = d.kv_attend(q, cache, table.to(DEV), put(lens), put(cu), max(new), max_len=max(lens), **kw)
    check(mixed, cache, q, table, lens, cu, **kw)
    # the single tokens by themselves
    one = [b for b, n in enumerate(new) if n == 1]
    rows = torch.tensor([cu[b] for b in one], device=DEV)
    alone = d.kv_attend(q[rows], cache, table[one].to(DEV), put([lens[b] for b in one]), **kw)
    check(alone, cache, q[rows], table[one], [lens[b] for b in one], list(range(len(one) + 1)), **kw)
