"""What a window hides of a branch of drafted tokens, from positions alone."""
import random

import pytest
import torch

decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")


def trees(new, seed, back):
    """(seen, depth, cu, parents) of random trees whose tokens go on from one of the `back` before them."""
    r = random.Random(seed)
    parents = [[r.randint(max(-1, i - back), i - 1) for i in range(n)] for n in new]
    made = [decode.tree(p) for p in parents]
    words = max(1, *(t[0].shape[1] for t in made))
    seen = torch.cat([torch.nn.functional.pad(t[0], (0, words - t[0].shape[1])) for t in made])
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return seen, torch.cat([t[1] for t in made]), torch.tensor(cu, dtype=torch.int32), parents


def row_bits(row):
    return {32 * w + i for w, x in enumerate(row.tolist()) for i in range(32) if x >> i & 1}


@pytest.mark.parametrize("window, sinks", [(1, 0), (2, 0), (5, 3), (7, 40), (33, 2), (64, 0), (10 ** 9, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("back", [1, 2, 6])
def test_a_branch_under_a_window(window, sinks, back):
    """Bits and context are those of the branch's own positions."""
    new, past = [70, 1, 0, 33, 9], [0, 2, 5, 38, 100]
    seen, depth, cu, parents = trees(new, window % 89 + back, back)
    got = decode.tree_window(seen, depth, cu, torch.tensor(past, dtype=torch.int32), window, sinks)
    assert got.dtype == torch.int32 and got.shape == seen.shape
    for b, n in enumerate(new):
        for i in range(n):
            branch, at = [], i
            while at >= 0:
                branch.append(at)
                at = parents[b][at]
            stands = past[b] + len(branch) - 1
            visible = lambda j: j > stands - window or j < sinks  # noqa: E731
            row = int(cu[b]) + i
            bits = row_bits(got[row])
            assert bits == {a for a in branch if visible(past[b] + int(depth[int(cu[b]) + a]))}
            # the position that kv_attend_tree takes from the bits shows the same of the context
            p = past[b] + len(bits - {i})
            assert [j > p - window or j < sinks for j in range(past[b])] == [visible(j) for j in range(past[b])]


def test_what_is_left_alone():
    seen, depth, cu, _ = trees([40, 3], 1, 3)
    past = torch.tensor([4, 9], dtype=torch.int32)
    assert torch.equal(decode.tree_window(seen, depth, cu, past, 0), seen)
    assert torch.equal(decode.tree_window(seen, depth, cu, past, int(depth.max()) + 1), seen)
    assert decode.tree_window(seen[:0], depth[:0], torch.zeros(3, dtype=torch.int32), past, 1).shape == (0, 2)
    for bad in ((-1, 0), (3, -1)):
        with pytest.raises(ValueError):
            decode.tree_window(seen, depth, cu, past, *bad)
