"""One decode step of a batch on a shared prompt, through the library's serving calls.

A prompt is written into the paged cache once; every request of the batch lists the
prompt's pages first in its block table and its own pages after them. A step then is
  smla.build_tables      pages and slots of the new tokens, from lengths on the GPU;
  smla.cache_append      their latent rows and indexer keys into the cache;
  smla.query_prep        their queries, rotated, and the indexer's, quantised;
  smla.shared_prefix_fwd attention over the prompt (read once for all) and own tokens,
  smla.sparse_mla_decode or, as the model's sparse layers do, over the top keys.
The projections that a model computes before and after are random numbers here.

    python examples/serve_step.py [--requests 64] [--prompt 16384] [--steps 4] [--kv fp8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import indexer_top_sparse_score_gb300 as smla  # noqa: E402
from indexer_top_sparse_score_gb300 import workloads  # noqa: E402

PAGE, ROPE, D_QK, D_V, D_IDX = 64, 64, 576, 512, 128


def rope_table(max_pos, device="cuda", theta=10000.0):
    """cos and sin of 32 angles per position, the angles in 64 bits."""
    inv = theta ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


class Batch:
    """A batch of requests on one prompt: cache, tables, lengths and weights."""

    def __init__(self, requests, prompt, max_own, heads=64, h_idx=32, topk=2048, kv="fp8", seed=0):
        assert prompt % PAGE == 0, "a shared prompt ends on a page: its pages are never written again"
        self.n, self.prompt, self.heads, self.h_idx, self.topk = requests, prompt, heads, h_idx, topk
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        own_pages = -(-max_own // PAGE)
        self.max_len = prompt + max_own
        pages = prompt // PAGE + requests * own_pages
        width, dtype = {"bf16": (D_QK, torch.bfloat16), "fp8": (D_QK, torch.uint8), "fp8_ds_mla": (656, torch.uint8)}[kv]
        new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.cache = workloads.Cache(new(pages, PAGE, width, dtype=dtype),
                                     new(pages, PAGE, dtype=torch.float32) if kv == "fp8" else None,
                                     new(pages, PAGE, D_IDX, dtype=torch.uint8), new(pages, PAGE, dtype=torch.float32), kv, "fp8")
        self.rope = rope_table(self.max_len)
        self.kv_norm = 1 + 0.1 * self._normal(D_V).float()
        self.k_norm, self.k_bias = 1 + 0.1 * self._normal(D_IDX).float(), 0.1 * self._normal(D_IDX).float()
        self.q_norm = 1 + 0.1 * self._normal(D_IDX).float()
        self.scale = 1 / math.sqrt(D_QK)
        free = torch.randperm(pages, generator=self.g, device="cuda").to(torch.int32)
        # the prompt, as a request of its own
        table = torch.full((1, self.max_len // PAGE + 1), -1, dtype=torch.int32, device="cuda")
        length = torch.full((1,), prompt, dtype=torch.int32, device="cuda")
        _, _, pos, slots, _, _, _ = smla.build_tables(torch.zeros_like(length), length, table, free, prompt)
        self._append(slots, pos)
        self.free = free[prompt // PAGE:].contiguous()
        # every request begins with the prompt's pages
        self.tables = table.expand(requests, -1).contiguous()
        self.lens = length.expand(requests).contiguous()

    def _normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def _append(self, slots, pos):
        return smla.cache_append(self.cache, slots, pos, self.rope, ckv=self._normal(slots.numel(), D_QK), kv_norm=self.kv_norm,
                                 k_idx=self._normal(slots.numel(), D_IDX), idx_norm=self.k_norm, idx_bias=self.k_bias)

    def step(self, new=1, sparse=True):
        """`new` more tokens for every request; (q, dense out, dense lse, sparse out or None)."""
        rows = self.n * new
        add = torch.full((self.n,), new, dtype=torch.int32, device="cuda")
        lens, _, pos, slots, _, used, ws = smla.build_tables(self.lens, add, self.tables, self.free, rows)
        ws_append = self._append(slots, pos)
        proj = self._normal(rows, self.heads, 192)  # each head's 128 values to be absorbed, and 64 to be rotated
        q = self._normal(rows, self.heads, D_QK)    # the absorbed part is in place; the rotated part comes next
        q, q_idx, w, ws_query = smla.query_prep(pos, self.rope, q_pe=proj[..., 128:], q=q, q_idx_raw=self._normal(rows, self.h_idx, D_IDX),
                                                w=torch.rand(rows, self.h_idx, generator=self.g, device="cuda"), idx_norm=self.q_norm,
                                                w_scale=D_IDX ** -0.5)
        out, lse, ws_dense = smla.shared_prefix_fwd(self.cache, self.tables, lens, self.max_len, self.prompt, new, q, self.scale)
        top = None
        checked = [ws, ws_append, ws_query, ws_dense]
        if sparse:
            top, _, _, ws_sparse = smla.sparse_mla_decode(self.cache, self.tables, lens, self.max_len, new, q, q_idx, w, self.topk,
                                                          self.scale)
            checked.append(ws_sparse)
        for w in checked:
            code, bits = smla.read_status(w)
            if code:
                raise smla.SmlaError(code, f"step (status bits {bits})")
        self.free = self.free[int(used):].contiguous()
        self.lens = lens
        return q, out, lse, top


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=64)
    p.add_argument("--prompt", type=int, default=16384)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--new", type=int, default=1, help="new tokens a request and step")
    p.add_argument("--kv", choices=["bf16", "fp8", "fp8_ds_mla"], default="fp8")
    a = p.parse_args(argv)
    smla.build()
    b = Batch(a.requests, a.prompt, max(PAGE, a.steps * a.new), kv=a.kv)
    for i in range(a.steps):
        _, out, lse, top = b.step(a.new)
        print(f"step {i}: {a.requests} requests at {int(b.lens[0])} tokens, |dense| {out.float().norm():.4f}, "
              f"|sparse| {top.float().norm():.4f}, lse {lse.mean():.4f}")


if __name__ == "__main__":
    main()
