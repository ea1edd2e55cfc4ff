"""kv_attend_tree where the most drafted tokens of a sequence is left out."""
import pytest
import torch

from drafts_ref import attend_tree, check_attend

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_kv_tree import make, put, trees  # noqa: E402


@pytest.mark.parametrize("new, words, G", [([16] * 16, 1, 4), ([32] * 40, 1, 8), ([5, 0, 33, 64, 2], 2, 2), ([3, 1], 4, 4)])
def test_a_batch_with_more_tokens_than_a_row_has_bits(new, words, G):
    """As README and the module's text call it: cu and seen alone."""
    lens = [n + 20 + 17 * i for i, n in enumerate(new)]
    cache, table, cu, q = make(lens, new, 2 * G, 2, 64, 16, torch.int8, torch.float16, len(new))
    bits = trees(new, 3, words=words)
    with decode.Decode() as d:
        got = d.kv_attend_tree(q, cache, table.cuda(), put(lens), bits, put(cu))
        check_attend(got, *attend_tree(q, cache, table, lens, bits, cu))
        with pytest.raises(ValueError, match="too few for max_q"):
            d.kv_attend_tree(q, cache, table.cuda(), put(lens), bits, put(cu), 32 * words + 1)
        with pytest.raises(ValueError, match="too few"):
            d.kv_attend_tree(q, cache, table.cuda(), put(lens), bits[:, :0], put(cu))


def test_one_token_each_takes_one_bit():
    lens = [5, 40]
    cache, table, _, q = make(lens, [1, 1], 4, 2, 64, 16, torch.int8, torch.float16, 1)
    with decode.Decode() as d:
        with pytest.raises(ValueError, match="too few"):
            d.kv_attend_tree(q, cache, table.cuda(), put(lens), torch.zeros((2, 0), dtype=torch.int32, device="cuda"))
