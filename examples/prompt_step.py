"""A step of prompts in the expanded form, through the library's calls.

Every request holds some context in the paged cache and gets a chunk of new tokens:
  smla.rope_table    the rotation table, once;
  smla.build_tables  pages and slots of the new tokens, from lengths on the GPU;
  smla.cache_append  their latent rows into the cache;
  smla.rope_apply    the rope part of their queries, in place;
  smla.cache_read    the new tokens' rows, and the context's a part at a time, back as bf16;
  (the model's up-projection turns latent rows into keys and values of each head: a plain product)
  smla.prompt_fwd    the new tokens among themselves, then each part of the context joined with
                     what is there.
The projections that a model computes before and after are random numbers here.

    python examples/prompt_step.py [--requests 4] [--context 3000] [--new 512] [--part 1024] [--kv fp8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import indexer_top_sparse_score_gb300 as smla  # noqa: E402
from indexer_top_sparse_score_gb300 import workloads  # noqa: E402

PAGE, D_QK, D_LAT, ROPE, D_NOPE, D_V, D_IDX = 64, 576, 512, 64, 128, 128, 128


class Prompts:
    """Requests that are being prefilled: cache, tables, lengths and weights."""

    def __init__(self, requests, max_len, heads=64, kv="fp8", seed=0):
        self.n, self.heads = requests, heads
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        width = -(-max_len // PAGE)
        pages = requests * width
        row, dtype = {"bf16": (D_QK, torch.bfloat16), "fp8": (D_QK, torch.uint8), "fp8_ds_mla": (656, torch.uint8)}[kv]
        new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.cache = workloads.Cache(new(pages, PAGE, row, dtype=dtype), new(pages, PAGE, dtype=torch.float32) if kv == "fp8" else None,
                                     new(pages, PAGE, D_IDX, dtype=torch.uint8), new(pages, PAGE, dtype=torch.float32), kv, "fp8")
        self.rope = smla.rope_table(max_len)
        self.kv_norm = 1 + 0.1 * self.normal(D_LAT).float()
        self.w_kv = (self.normal(D_LAT, heads * (D_NOPE + D_V)).float() / math.sqrt(D_LAT)).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(D_NOPE + ROPE)
        self.free = torch.randperm(pages, generator=self.g, device="cuda").to(torch.int32)
        self.tables = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def expand(self, starts, cu, rows):
        """Keys without their rope part, values and the rope part of `rows` packed rows of the cache."""
        latent, pe, _, ws = smla.cache_read(self.cache, self.tables, cu, rows, starts=starts)
        kv = (latent @ self.w_kv).view(rows, self.heads, D_NOPE + D_V)
        return kv[..., :D_NOPE], kv[..., D_NOPE:], pe, ws

    def step(self, new, part=1024):
        """new[b] more tokens for request b; (rotated queries, out, lse) of the packed new tokens."""
        add = torch.tensor(new, dtype=torch.int32, device="cuda")
        rows = sum(new)
        lens, cu, pos, slots, _, used, ws = smla.build_tables(self.lens, add, self.tables, self.free, rows)
        checked = [ws, smla.cache_append(self.cache, slots, pos, self.rope, ckv=self.normal(rows, D_QK), kv_norm=self.kv_norm)]
        q = self.normal(rows, self.heads, D_NOPE + ROPE)
        _, ws = smla.rope_apply(q[..., D_NOPE:], pos, self.rope, out=q[..., D_NOPE:])
        checked.append(ws)
        k, v, pe, ws = self.expand(self.lens, cu, rows)
        checked.append(ws)
        out, lse, ws = smla.prompt_fwd(q, k, v, cu, cu, self.scale, k_pe=pe, out_dtype=torch.float32)
        checked.append(ws)
        context = self.lens.tolist()
        for a in range(0, max(context), part):  # the same part of every request's context at a time
            held = [max(0, min(c, a + part) - a) for c in context]
            starts = torch.full((self.n,), a, dtype=torch.int32, device="cuda")
            cu_k = torch.tensor([0] + held, device="cuda").cumsum(0).to(torch.int32)
            k, v, pe, ws = self.expand(starts, cu_k, sum(held))
            checked.append(ws)
            out, lse, ws = smla.prompt_fwd(q, k, v, cu, cu_k, self.scale, k_pe=pe, causal=False, prev_out=out, prev_lse=lse, out=out, lse=lse)
            checked.append(ws)
        for w in checked:
            code, bits = smla.read_status(w)
            if code:
                raise smla.SmlaError(code, f"step (status bits {bits})")
        self.free = self.free[int(used):].contiguous()
        self.lens = lens
        return q, out, lse


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--context", type=int, default=3000)
    p.add_argument("--new", type=int, default=512, help="new tokens a request")
    p.add_argument("--part", type=int, default=1024, help="tokens of a request's context that are expanded at a time")
    p.add_argument("--kv", choices=["bf16", "fp8", "fp8_ds_mla"], default="fp8")
    a = p.parse_args(argv)
    smla.build()
    b = Prompts(a.requests, a.context + a.new, kv=a.kv)
    for i, new in enumerate((a.context, a.new)):
        _, out, lse = b.step([new] * a.requests, a.part)
        print(f"step {i}: {a.requests} requests at {int(b.lens[0])} tokens, |out| {out.norm():.4f}, lse {lse.mean():.4f}")


if __name__ == "__main__":
    main()
