"""kv_attend_tree with many rows: parts of items over more row blocks than lanes, a full workspace, and more items than
joins (tree_cases), against attention over each row's own tokens in float64."""
import pytest
import torch

import tree_cases
from drafts_ref import attend_tree, check_attend

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_kv_tree import E4M3, make, put, trees  # noqa: E402

BY_NAME = {c[0]: c for c in tree_cases.CASES}


@pytest.mark.parametrize("code, dtype, window, sinks", [(torch.int8, torch.float16, 0, 0), (E4M3, torch.bfloat16, 3000, 70)])
@pytest.mark.parametrize("name", list(BY_NAME))
def test_against_the_definition(name, code, dtype, window, sinks):
    _, lens, new, G, H, D, page = BY_NAME[name]
    cache, table, cu, q = make(lens, new, G * H, H, D, page, code, dtype, len(name))
    bits, out = trees(new, 5), torch.full_like(q, 7)
    with decode.Decode() as d:
        d.kv_attend_tree(q, cache, table.cuda(), put(lens), bits, put(cu), max(new), max_len=max(lens), window=window, sinks=sinks, out=out)
        ref, bound = attend_tree(q, cache, table, lens, bits, cu, window, sinks)
        check_attend(out, ref, bound)
        again = d.kv_attend_tree(q, cache, table.cuda(), put(lens), bits, put(cu), max(new), max_len=max(lens), window=window, sinks=sinks)
        assert torch.equal(again, out)
