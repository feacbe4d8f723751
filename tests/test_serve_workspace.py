"""The workspace of the shared-prompt attention (no GPU): its size, and the slots of the partial results where
nothing is shared (piece_slot of prefix.cu), on the model of how the work is cut."""
import random

import pytest

import indexer_top_sparse_score_gb300 as smla
from test_prefix_partition import COSTS, pieces


@pytest.mark.parametrize("kv", [smla.SMLA_BF16, smla.SMLA_FP8_E4M3, smla.SMLA_FP8_DS_MLA])
def test_size_does_not_grow_with_the_rows_of_a_prompt_chunk(kv):
    smla.build()
    size = lambda tokens, n=1: smla.lib().smla_shared_prefix_fwd_workspace_size(n, 65536, 0, tokens, 64, kv)  # noqa: E731
    assert size(8192) < 64 << 20 and size(16384) < 64 << 20 and size(2, 4000) < 64 << 20
    assert size(16384) - size(8192) <= 8 * 4096  # where each segment starts on the line
    assert size(1) <= size(128) <= size(8192)


@pytest.mark.parametrize("seed", range(40))
def test_two_slots_a_pair_hold_the_cut_pieces(seed):
    r = random.Random(seed)
    pairs = r.choice([1, 2, 7, 76])
    tiles = [r.choice([0, 1, 2, r.randrange(1, 300)]) for _ in range(r.choice([pairs + 1, 90, 600]))]
    got, start, _, _ = pieces(tiles, 0, COSTS[seed % len(COSTS)], pairs)
    cut = [(2 * p + (t0 == 0), s) for (s, p), (t0, t1) in got.items() if (t0, t1) != (0, tiles[s])]
    assert len({slot for slot, _ in cut}) == len(cut) and all(0 <= slot < 2 * pairs for slot, _ in cut)
    whole = {s for (s, p), t in got.items() if t == (0, tiles[s])}
    assert whole.isdisjoint(s for _, s in cut)  # a segment's results come from one place
    assert whole | {s for _, s in cut} == {s for s, t in enumerate(tiles) if t}
