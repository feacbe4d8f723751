"""Long requests and cut keys on the GPU with the bounds of prompt_tiles, which no lost or doubled key tile passes."""
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import prompt_common as pc
import prompt_tiles as pt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


SHAPES = [([2, 70], [140000, 300], 1, 1), ([1], [40000], 1, 1), ([1, 2], [20011, 9000], 16, 16), ([5], [30000], 16, 1), ([300], [20000], 4, 4),
          ([1] * 9, [5000 + 777 * i for i in range(9)], 8, 2), ([1] * 9, [5000 + 777 * i for i in range(9)], 16, 16), ([257, 0, 513, 3], [257, 900, 513, 3], 2, 2),
          ([900, 40], [900, 2000], 12, 4), ([60], [60], 16, 16), ([7, 2], [4, 1000], 4, 1)]


@pytest.mark.parametrize("by", ["tile", "key"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,heads,kv_heads", SHAPES)
def test_prompt_counts(ql, kl, heads, kv_heads, causal, by):
    q, k, v, cq, ck = pt.count_case(ql, kl, heads, kv_heads, 192, by, seed=60)
    out, lse, ws = smla.prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), 0.07, causal=causal, out_dtype=torch.float32)
    assert smla.read_status(ws)[0] == 0
    pt.check_counts(out[:sum(ql)], lse[:sum(ql)], *pt.counts(ql, kl, causal, by))


def test_prompt_counts_of_more_requests_than_the_plans_threads():
    ql, kl = [i % 4 for i in range(2500)], [i % 4 + i % 5 for i in range(2500)]
    kl[1200], kl[2499] = 30000, 5000
    q, k, v, cq, ck = pt.count_case(ql, kl, 2, 1, 192, "key", seed=61)
    out, lse, ws = smla.prompt_fwd(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), 0.07, out_dtype=torch.float32)
    assert smla.read_status(ws)[0] == 0
    pt.check_counts(out, lse, *pt.counts(ql, kl, True, "key"))


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,heads,kv_heads", SHAPES[:6])
def test_prompt_rows(ql, kl, heads, kv_heads, causal, fp32):
    q, k, v, pe, cq, ck = (t.cuda() for t in pc.prompt_case(ql, kl, heads, kv_heads, 192, True, seed=62))
    out, lse, ws = smla.prompt_fwd(q, k, v, cq, ck, 192 ** -0.5, k_pe=pe, causal=causal, out_dtype=torch.float32 if fp32 else torch.bfloat16)
    assert smla.read_status(ws)[0] == 0
    pt.check_rows(out, lse, pc.prompt_reference(q, k, v, pe, cq, ck, 192 ** -0.5, causal))
