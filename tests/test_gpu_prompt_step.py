"""The expanded-prompt calls together, as examples/prompt_step.py runs them."""
import os
import sys

import pytest
import torch

import prompt_common as pc
import serve_common as sc

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp8_ds_mla"])
def test_steps_against_the_reference(kv):
    """Three chunks, ragged and idle requests among them, in parts of 100 tokens of context: against 64 bits over keys and
    values that are expanded (and rounded to bf16, as the step does) from what the cache holds."""
    import prompt_step
    heads = 4
    b = prompt_step.Prompts(3, 500, heads=heads, kv=kv, seed=5)
    held = [0, 0, 0]
    for new in ([130, 1, 64], [3, 0, 200], [70, 99, 1]):
        q, out, lse = b.step(new, part=100)
        latent = torch.from_numpy(sc.latent_values(b.cache.to("cpu"))).cuda().to(torch.bfloat16)
        rows = torch.cat([b.tables[i, torch.arange(h + a, device="cuda") // 64].long() * 64 + torch.arange(h + a, device="cuda") % 64
                          for i, (h, a) in enumerate(zip(held, new))])
        kept = latent[rows]
        kv_rows = (kept[:, :512] @ b.w_kv).view(-1, heads, 256)
        held = [h + a for h, a in zip(held, new)]
        ref = pc.prompt_reference(q, kv_rows[..., :128], kv_rows[..., 128:], kept[:, 512:], pc.cu(new), pc.cu(held), b.scale, True)
        # The product of latent rows may be rounded to the other bf16 neighbour where it is taken over other rows at a time
        # (sums of 512 products in fp32 in another order): a step of 2^-7 on few values, of keys and values of 128.
        # So rows are compared as wholes: each differing value moves a logit by 2^-7 |q k| / sqrt(192), far under
        # the 2^-8 of a probability, and a row by less than its rounding.
        err = (out.double() - ref[0]).norm(dim=-1) / ref[0].norm(dim=-1)
        assert err.max() <= 2.0 ** -7 and (lse.double() - ref[1]).abs().max() <= 2.0 ** -7
    assert b.lens.tolist() == held == [203, 100, 265]


def test_example_runs(capsys):
    import prompt_step
    prompt_step.main(["--requests", "2", "--context", "300", "--new", "100", "--part", "128"])
    assert capsys.readouterr().out.count("step") == 2
    torch.cuda.synchronize()
