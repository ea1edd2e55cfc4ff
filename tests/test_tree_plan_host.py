"""The GPU tests of kv_attend_tree with many rows reach what they are for."""
import pytest

import tree_cases
from tree_plan import JOINS, many_rows, plan

BY_NAME = {c[0]: c for c in tree_cases.CASES}


@pytest.mark.parametrize("name", list(BY_NAME))
def test_cases_reach_their_paths(name):
    _, lens, new, G, H, D, _ = BY_NAME[name]
    assert many_rows(new, G, D)
    p = plan(lens, new, G, H, D)
    here, there = p.parts[:64], p.parts[64:]
    if name.startswith("uneven"):
        assert len(p.parts) > 128
        for side in (here, there):
            assert any(n > 1 for n in side) and any(n == 1 for n in side) and any(n == 0 for n in side)
    if name == "long 0":
        assert all(n > 1 for n in here) and all(n == 1 for n in there)
    if name == "long 64":
        assert all(n == 1 for n in here) and all(n > 1 for n in there)
    assert p.again == name.startswith("room")
    assert (len(p.parts) * H > JOINS) == (name == "many items")
