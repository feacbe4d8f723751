"""Attention cases whose answers a lost or doubled key changes visibly, however many keys there are.

Counts: all logits are 0, so every probability before the division is exactly 1, every sum a whole number below 2^24
(exact in fp32), and lse = ln(keys seen). V holds ones: key j's in column j // 128 mod 128 (by tile) or in column
j mod 128 (by key), so that out * keys is how many keys of each kind were seen.
Rows: random keys and values, each row's error as a vector against its length."""
import math

import torch

import prompt_common as pc


def count_case(ql, kl, heads, kv_heads, d, by, seed=0):
    """(q, k, v, cu_q, cu_k) without a rope part; random queries, keys of zeros."""
    q, k, v, _, cq, ck = pc.prompt_case(ql, kl, heads, kv_heads, d, False, seed=seed)
    k, v = torch.zeros_like(k), torch.zeros_like(v)
    for b, n in enumerate(kl):
        j = torch.arange(n)
        v[int(ck[b]) + j, :, (j // 128 if by == "tile" else j) % 128] = 1.0
    return q, k, v, cq, ck


def counts(ql, kl, causal, by):
    """Keys of each kind that every row sees, and their number: [rows, 128] and [rows] float64."""
    out, n = [], []
    for nq, nk in zip(ql, kl):
        j = torch.arange(nk)
        kind = (j // 128 if by == "tile" else j) % 128
        upto = torch.zeros(nk + 1, 128, dtype=torch.float64)
        upto[1:] = torch.nn.functional.one_hot(kind, 128).double().cumsum(0)
        seen = (torch.arange(nq) + nk - nq + 1).clamp(0, nk) if causal else torch.full((nq,), nk)
        out.append(upto[seen])
        n.append(seen.double())
    return torch.cat(out), torch.cat(n)


def check_counts(out, lse, count, seen):
    """out [rows, heads, 128] fp32: a whole number times a reciprocal, and perhaps a part's weight of exactly 1: four
    roundings at most of 2^-24, the reciprocal's among them. lse: a logarithm to 2^-21 and two products."""
    out, lse = out.double().cpu(), lse.double().cpu()
    want = torch.where(seen[:, None] > 0, count / seen.clamp_min(1)[:, None], 0.0)[:, None]
    assert ((out - want).abs() <= 4 * pc.FP32 * want).all(), f"counts off by {float(((out - want).abs() * seen[:, None, None]).max())} keys"
    some = seen > 0
    assert lse[~some].isneginf().all()
    ln = seen[some].log()[:, None]
    assert ((lse[some] - ln).abs() <= 2.0 ** -21 * (1 + ln)).all(), f"lse off by {float((lse[some] - ln).abs().max())}"


def check_rows(out, lse, ref):
    """Probabilities are rounded to bf16, each off by at most 2^-8 of itself and about 2^-8 / sqrt(3) in the mean
    square, whichever way: a row, whose length is that of its products with independent values put together at random, is
    off by 2^-8 / sqrt(3) of its length; rounding it to bf16 adds as much. Together 0.0032; 2^-7 = 0.0078 is over twice that (the spread
    over 128 columns is some 6%). A tile of 128 keys of n is sqrt(128 / n) of the length: 0.03 of 140,000.
    lse: probabilities to 2^-21 each and a rounding of 2^-24 a tile (1,100 tiles: 2^-14 if all went one way, 2^-19 at random):
    2^-16. A tile of 140,000 keys is 2^-10."""
    ro, rl = ref[0], ref[1]
    out, lse = out.double().to(ro.device), lse.double().to(ro.device)
    some = ~rl.isneginf()
    assert torch.equal(~lse.isneginf(), some) and (out[~some] == 0).all()
    err = (out - ro).norm(dim=-1)[some] / ro.norm(dim=-1)[some]
    assert err.max() <= 2.0 ** -7, f"rows off by {float(err.max())} of their length"
    off = (lse - rl)[some].abs() - 2.0 ** -21 * rl[some].abs()
    assert off.max() <= 2.0 ** -16, f"lse off by {float(off.max())}"


def exact_row(n, seed=0):
    """One row over n random keys on the CPU in float64: (probabilities, values)."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, generator=g, dtype=torch.float64) * math.sqrt(0.9)
    return (z - z.max()).exp(), torch.randn(n, 128, generator=g, dtype=torch.float64)
