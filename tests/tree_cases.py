"""Calls of kv_attend_tree with many rows: (name, lens, drafts, query heads to a key-value head, key-value heads, channels, page size)."""
import random


def _case(name, context, new, G, H, D, page):
    return name, [c + n for c, n in zip(context, new)], new, G, H, D, page


def _cases():
    r = random.Random(7)
    # more row blocks than lanes, the long sequences on both sides of the 64th
    for D, H, page in ((128, 2, 16), (64, 2, 16), (256, 1, 32)):
        n = [r.randint(0 if D == 128 else 15, 40) for _ in range(100)]
        n[3] = n[80] = n[95] = 40 if D != 256 else 70
        context = [r.choice((0, 5, 200, 900)) for _ in n]
        context[3], context[80], context[95] = 6000, 20000, 9000
        yield _case(f"uneven {D}", context, n, 8, H, D, page)
    # none of the first 64 has parts, and all of them
    for at in (range(64), range(64, 100)):
        n = [r.randint(10, 32) for _ in range(100)]
        yield _case(f"long {at[0]}", [9000 if i in at else 100 for i in range(100)], n, 8, 1, 128, 64)
    # so many items of two parts that the workspace does not hold them
    for D, n, H in ((128, 100, 4), (256, 25, 4)):
        yield _case(f"room {D}", [r.randint(9000, 10000) for _ in range(n)], [32 if D == 128 else 64] * n, 8, H, D, 64)
    # more items than the list of joins holds
    n = [r.randint(9, 12) for _ in range(129)]
    yield _case("many items", [r.choice((3, 70, 400)) if i != 70 else 9000 for i in range(129)], n, 8, 8, 128, 64)


CASES = list(_cases())
