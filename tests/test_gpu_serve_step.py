"""The serving calls together, as examples/serve_step.py runs them."""
import os
import sys

import pytest
import torch

import serve_common as sc

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp8_ds_mla"])
def test_steps_against_the_reference(kv):
    """Three steps across a page border: the dense attention against 64 bits over what the cache holds, and
    (all keys are within the top-k) the sparse attention of the same step against the same."""
    import serve_step
    b = serve_step.Batch(5, 640, 192, heads=64, topk=1024, kv=kv, seed=3)
    for new in (63, 2, 5):
        q, out, lse, top = b.step(new, sparse=new <= 8)
        ref = sc.attention_reference(b.cache.to("cpu"), b.tables.cpu(), b.lens.cpu(), new, q.cpu(), 640, sc.SM_SCALE)
        sc.check_attention(out, lse, ref, kv)
        if top is not None:
            assert (top.float() - out.float()).norm() <= 1e-2 * out.float().norm()
    assert b.lens.tolist() == [640 + 70] * 5
    own = b.tables[:, 10:12]
    assert (own >= 0).all() and own.flatten().unique().numel() == 10  # pages of their own
    assert (b.tables[:, :10] == b.tables[0, :10]).all() and (b.tables[:, 12:] == -1).all()


def test_example_runs(capsys):
    import serve_step
    serve_step.main(["--requests", "3", "--prompt", "128", "--steps", "2", "--new", "2"])
    assert capsys.readouterr().out.count("step") == 2
    torch.cuda.synchronize()
