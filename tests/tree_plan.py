"""How kv_attend_tree cuts a call with many rows into parts, by the rules of decode/attend.hip and attend_tile.hip on 256 compute units."""
from typing import NamedTuple

CUS, STAGE, LEAST, JOINS, WORKSPACE = 256, 64, 4, 1024, 64 << 20


class Plan(NamedTuple):
    parts: list     # of each (sequence, row block) and head; 0 where there are no rows
    again: bool     # whether the first choice had more parts than the workspace holds
    room: int


def up(a, b):
    return -(-a // b)


def many_rows(new, G, D):
    """Whether the kernel for many rows takes the call."""
    rows, mean = G * max(new), G * sum(new) // len(new)
    if rows <= 64:
        return False
    return mean > 150 if D == 64 else mean > 68 if D == 128 else rows > 511 or 5 * mean > 3 * rows


def plan(lens, new, G, H, D):
    block = 128 if D == 256 else 256
    blocks = up(G * max(new), block)
    tiles = [up(n, STAGE) if G * q > i * block and n > 0 else int(G * q > i * block) for n, q in zip(lens, new) for i in range(blocks)]
    items, room = len(tiles) * H, WORKSPACE // (4 * block * (D + 2))
    if items > JOINS:
        return Plan([min(t, 1) for t in tiles], False, room)
    total, most = sum(tiles) * H, max(tiles)
    until = lambda chunk, parts: chunk + 3 if parts <= CUS else (total + 3 * parts) / CUS + chunk / 2  # noqa: E731
    chunk_of = lambda want: min(most, max(LEAST, up(total, want)))  # noqa: E731
    chunk, least = most, until(most, items)
    for rounds in (2, 1):
        c = chunk_of(rounds * CUS)
        u = until(c, total / c + (0 if rounds == 1 else items)) + 4
        if u < least:
            chunk, least = c, u
    cut = lambda chunk: [max(1, up(t, chunk)) if t else 0 for t in tiles]  # noqa: E731
    many = lambda parts: sum(p for p in parts if p > 1) * H  # noqa: E731
    again = many(cut(chunk)) > room
    if again:
        chunk = chunk_of(min(CUS, room // 2))
    assert many(cut(chunk)) <= room and sum(max(p, 1) for p in cut(chunk)) * H <= items + 2 * CUS
    return Plan(cut(chunk), again, room)
