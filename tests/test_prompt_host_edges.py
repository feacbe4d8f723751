"""Refusals of the expanded-prompt calls beyond test_prompt_host (no GPU: the fake pointers are never dereferenced)."""
import itertools

import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
from test_prompt_host import FAKE, INVALID, L, WORKSPACE, _rope  # noqa: F401


# ---------------------------------------------------------------------------- places of the rotated heads
def _shares(rows, row, heads, head, dim):
    at = sorted(i * row + h * head for i, h in itertools.product(range(rows), range(heads)))
    return any(b - a < dim for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("dim", [8, 64])
@pytest.mark.parametrize("rows,heads", [(1, 1), (2, 2), (5, 4), (3, 7), (9, 2)])
def test_rope_refuses_outputs_whose_heads_share_values(L, rows, heads, dim):  # noqa: F811
    """Every pair of strides up to some rows' length, against all places: only those that overlap are refused (here by their
    code; the others come as far as the missing workspace)."""
    for row in range(dim, dim * (2 * heads + 2) + 1, max(8, dim // 4)):
        for head in range(dim, dim * (2 * rows + 2) + 1, max(8, dim // 4)):
            for place in (dict(xr=row, xh=head, out=FAKE), dict(xr=heads * dim, xh=dim)):  # in place or not
                rc = _rope(L, rows=rows, h=heads, dim=dim, outr=row, outh=head, ws=None, **place)
                assert rc == (INVALID if _shares(rows, row, heads, head, dim) else WORKSPACE), (row, head)


def test_rope_accepts_large_strides(L):  # noqa: F811
    big = 1 << 60
    assert _rope(L, rows=1 << 30, h=1 << 10, outr=64 << 10, outh=64, ws=None) == WORKSPACE
    assert _rope(L, rows=1 << 30, h=1 << 10, outr=64, outh=64 << 30, ws=None) == WORKSPACE
    assert _rope(L, rows=1 << 30, h=1 << 10, outr=64, outh=64, ws=None) == INVALID
    assert _rope(L, rows=1 << 30, h=1 << 20, outr=big, outh=big, ws=None) == INVALID


def test_view_of_a_cache_without_indexer_keys():
    """As the C calls take it: no keys, no width."""
    class Dense:
        kv, kv_scale, kv_dtype = torch.zeros(3, 64, 576, dtype=torch.bfloat16), None, "bf16"
        k_idx = k_idx_scale = idx_dtype = None

    c = smla.make_cache(Dense())
    assert c.kv == Dense.kv.data_ptr() and not c.k_idx and c.d_idx == 0 and c.num_pages == 3 and c.page_size == 64
