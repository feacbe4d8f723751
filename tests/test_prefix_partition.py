"""How the shared-prompt attention cuts its work, as a model on the CPU: segments
(128 rows x a range of key tiles) lie one after another on a line, pair i of P
walks the i-th of P equal stretches. Every tile has to be walked once, every
piece has to have a slot of its own inside the workspace, and the joining step
has to find exactly the pieces of a segment."""
import random

import pytest

OVERHEAD = 6


def pieces(tiles, pairs):
    """{(segment, pair): (t0, t1)} as the kernel walks them, and {segment: start}."""
    cost = [t + OVERHEAD if t else 0 for t in tiles]
    total = sum(cost)
    got, start = {}, {}
    for p in range(pairs):
        x, y = total * p // pairs, total * (p + 1) // pairs
        if x == y:
            continue
        s = a = 0
        while a + cost[s] <= x:  # the segment that holds x
            a += cost[s]
            s += 1
        while s < len(tiles) and a < y:
            if cost[s]:
                if a >= x:
                    assert s not in start
                    start[s] = a
                t0, t1 = max(x - a - OVERHEAD, 0), min(y - a - OVERHEAD, tiles[s])
                if t1 > t0:
                    got[s, p] = (t0, t1)
                a += cost[s]
            s += 1
    return got, start, total


def joined(s, start, tiles, total, pairs):
    """The pairs whose pieces the joining step reads for segment s."""
    t0 = start[s] + OVERHEAD
    t1 = t0 + tiles[s]
    return [q for q in range(pairs) if max(total * q // pairs, t0) < min(total * (q + 1) // pairs, t1)]


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_once_and_every_piece_found(seed):
    r = random.Random(seed)
    pairs = r.choice([1, 2, 7, 76])
    tiles = [r.choice([0, 1, 2, r.randrange(1, 300)]) for _ in range(r.choice([1, 2, 5, 60, 300]))]
    got, start, total = pieces(tiles, pairs)
    slots = [s + p for s, p in got]
    assert len(set(slots)) == len(slots) and all(0 <= v < len(tiles) + pairs for v in slots)
    for s, n in enumerate(tiles):
        mine = sorted((t, q) for (i, q), t in got.items() if i == s)
        assert [t for (a, b), _ in mine for t in range(a, b)] == list(range(n))
        if n:
            assert joined(s, start, tiles, total, pairs) == [q for _, q in mine]
    loads = [sum(t1 - t0 for (s, q), (t0, t1) in got.items() if q == p) for p in range(pairs)]
    if total >= pairs:
        assert max(loads) <= total / pairs + 1
    for a in range(0, len(tiles) - 1):  # two segments of one row: never more pieces than pairs + 2
        b = r.randrange(a + 1, len(tiles))
        if tiles[a] and tiles[b]:
            n = len(joined(a, start, tiles, total, pairs)) + len(joined(b, start, tiles, total, pairs))
            assert n <= pairs + 2
