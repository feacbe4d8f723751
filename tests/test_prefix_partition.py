"""How the shared-prompt attention cuts its work, as a model on the CPU: segments
(128 rows x a range of key tiles) lie one after another on a line, where each start
of a segment and each tile has a cost; pair i of P walks the tiles that begin in the
i-th of P equal stretches. Every tile has to be walked once, every
piece has to have a slot of its own inside the workspace, and the joining step
has to find exactly the pieces of a segment."""
import random

import pytest

COSTS = [(20, 4, 4), (40, 4, 7), (34, 4, 10), (34, 10, 10)]  # start, shared tile, own tile


def stretch(cost, one, tiles, a, x, y):
    up = lambda v: -(-max(v, 0) // one)  # noqa: E731
    return up(x - a - cost[0]), min(up(y - a - cost[0]), tiles)


def pieces(tiles, n_shared, cost, pairs):
    """{(segment, pair): (t0, t1)} as the kernel walks them, and {segment: start}."""
    one = [cost[1] if s < n_shared else cost[2] for s in range(len(tiles))]
    whole = [cost[0] + t * o if t else 0 for t, o in zip(tiles, one)]
    total = sum(whole)
    got, start = {}, {}
    for p in range(pairs):
        x, y = total * p // pairs, total * (p + 1) // pairs
        if x == y:
            continue
        s = a = 0
        while a + whole[s] <= x:  # the segment that holds x
            a += whole[s]
            s += 1
        while s < len(tiles) and a < y:
            if whole[s]:
                t0, t1 = stretch(cost, one[s], tiles[s], a, x, y)
                if t1 > t0:
                    got[s, p] = (t0, t1)
                    if t0 == 0:  # the pair with the first tile says where the segment starts
                        assert s not in start
                        start[s] = a
                a += whole[s]
            s += 1
    return got, start, total, one


def joined(s, start, tiles, cost, one, total, pairs):
    """The pairs whose pieces the joining step reads for segment s."""
    got = []
    for q in range(pairs):
        t0, t1 = stretch(cost, one[s], tiles[s], start[s], total * q // pairs, total * (q + 1) // pairs)
        if t1 > t0:
            got.append(q)
    return got


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_once_and_every_piece_found(seed):
    r = random.Random(seed)
    cost = COSTS[seed % len(COSTS)]
    pairs = r.choice([1, 2, 7, 76])
    n = r.choice([1, 2, 5, 60, 300])
    n_shared = r.choice([0, n // 2])
    tiles = [r.choice([0, 1, 2, r.randrange(1, 300)]) for _ in range(n)]
    got, start, total, one = pieces(tiles, n_shared, cost, pairs)
    slots = [s + p for s, p in got]
    assert len(set(slots)) == len(slots) and all(0 <= v < len(tiles) + pairs for v in slots)
    for s, k in enumerate(tiles):
        mine = sorted((t, q) for (i, q), t in got.items() if i == s)
        assert [t for (a, b), _ in mine for t in range(a, b)] == list(range(k))
        if k:
            assert joined(s, start, tiles, cost, one, total, pairs) == [q for _, q in mine]
    loads = [sum((t1 - t0) * one[s] for (s, q), (t0, t1) in got.items() if q == p) for p in range(pairs)]
    if total >= pairs:
        assert max(loads) <= total / pairs + max(one) + 1
    for a in range(0, len(tiles) - 1):  # two segments of one row: never more pieces than pairs + 2
        b = r.randrange(a + 1, len(tiles))
        if tiles[a] and tiles[b]:
            both = sum(len(joined(i, start, tiles, cost, one, total, pairs)) for i in (a, b))
            assert both <= pairs + 2
