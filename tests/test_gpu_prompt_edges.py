"""Calls at the edges of what include/smla_prompt.h allows, on the GPU."""
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import prompt_common as pc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


# ---------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("lead", [16, 32, 48])
@pytest.mark.parametrize("ql,kl", [([2, 1, 5], [9000, 3, 17000]), ([300], [5000]), ([70, 9], [90, 20])])
def test_prompt_workspace_on_any_16_byte_boundary(lead, ql, kl):
    """Cut keys (partial results in the workspace), uncut ones, a call without a plan: the bits that the allocator's own
    boundary gives, and nothing written behind the size that the call asks for."""
    q, k, v, pe, cq, ck = (t.cuda() for t in pc.prompt_case(ql, kl, 4, 4, 192, True, seed=50))
    need = smla.prompt_workspace_bytes(sum(ql), sum(kl), len(ql), 4, 4)
    call = lambda ws: smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, ws=ws)  # noqa: E731
    out, lse, _ = call(smla.workspace(need))
    raw = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws = raw[lead:lead + need]
    assert ws.data_ptr() % 64 == lead % 64
    got, glse, _ = call(ws)
    assert smla.read_status(ws)[0] == 0
    assert torch.equal(got, out) and torch.equal(glse, lse)
    assert (raw[:lead] == 171).all() and (raw[lead + need:] == 171).all()
