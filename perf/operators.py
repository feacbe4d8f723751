"""Measured cases of the serving operators around the paged latent cache.

Four operators that a serving step with many requests on one long common prompt runs in this order:
  tables     block tables and slot maps built on the GPU from the requests' lengths;
  append     norm, rotation, quantisation and paged write of the new tokens' latent and indexer-key rows;
  query      rotation of the attention queries, norm + rotation + quantisation of each indexer head's query;
  attention  attention of every request's new tokens over the prompt all of them share (computed once for
             all) and over each request's own tokens.
`run` computes them with elementary torch operations (own = False) or through the package (own = True).
"""
import math

import torch

own = False

PAGE, D_QK, D_V, ROPE = 64, 576, 512, 64
IDX_H, IDX_D = 32, 128
EPS = 1e-6
MAX_POS = 1 << 17
DS_BYTES = 656


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of the decode batch: 64 requests of 8K-128K tokens, 2 new tokens each
        dict(name="tables decode 64x2", op="tables", n_seqs=64, new_min=2, new_max=2, ctx_min=8192, ctx_max=131000),
        # a mixed step: many requests, some idle, some with long ragged chunks of prompt
        dict(name="tables mixed 1000", op="tables", n_seqs=1000, new_min=0, new_max=257, ctx_min=0, ctx_max=16001),
        # the decode batch's 128 new rows into the FP8 cache
        dict(name="append fp8 128", op="append", rows=128, kv="fp8", idx="fp8", holes=False),
        # one 8,192-token prefill chunk into the BF16 cache
        dict(name="append bf16 8192", op="append", rows=8192, kv="bf16", idx="fp8", holes=False),
        # an odd, padded batch into the 656-byte rows
        dict(name="append ds_mla 5003", op="append", rows=5003, kv="fp8_ds_mla", idx="fp8", holes=True),
        # the queries of the decode batch, and of one prefill chunk
        dict(name="query 128", op="query", rows=128, heads=64),
        dict(name="query 8192", op="query", rows=8192, heads=64),
        # the smallest call: one request, one token, a short odd context
        dict(name="attention 1x1 1K", op="attention", n_seqs=1, q=1, heads=64, kv="bf16", shared=1001, own_min=99, own_max=99),
        # 16 heads, odd counts, a shared prompt that ends inside a page
        dict(name="attention 37x2 5K h16", op="attention", n_seqs=37, q=2, heads=16, kv="fp8_ds_mla", shared=5003, own_min=66, own_max=901),
        # an ordinary decode batch on a 16K prompt, FP8 cache
        dict(name="attention 64x2 16K fp8", op="attention", n_seqs=64, q=2, heads=64, kv="fp8", shared=16384, own_min=8, own_max=2048),
        # the largest: the decode batch on a 64K prompt, BF16 cache
        dict(name="attention 64x2 64K", op="attention", n_seqs=64, q=2, heads=64, kv="bf16", shared=65536, own_min=64, own_max=4096),
        # a chunk of prompt: 1,024 tokens of one request after 8,192 cached ones
        dict(name="attention 1x1024 8K", op="attention", n_seqs=1, q=1024, heads=64, kv="bf16", shared=8192, own_min=1024, own_max=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "query", "attention", "attention", "attention"])
    if op == "tables":
        lo = rng.choice([0, 1])
        return dict(op=op, n_seqs=_log(rng, 1, 1000), new_min=lo, new_max=lo + _log(rng, 1, 256), ctx_min=rng.randrange(0, 64),
                    ctx_max=_log(rng, 64, 16000))
    if op == "append":
        return dict(op=op, rows=_log(rng, 1, 8192), kv=rng.choice(["bf16", "fp8", "fp8_ds_mla"]), idx=rng.choice(["fp8", "bf16"]),
                    holes=rng.random() < 0.5)
    if op == "query":
        return dict(op=op, rows=_log(rng, 1, 8192), heads=rng.choice([16, 64]))
    while True:
        q = rng.choice([1, 1, 2, 3, 4, _log(rng, 1, 512)])
        n = _log(rng, 1, 64) if q <= 8 else 1
        kv = rng.choice(["bf16", "fp8", "fp8_ds_mla"])
        least = q + (PAGE if kv == "fp8_ds_mla" else 0)  # contexts kept in the tile-scaled rows have a page at least
        c = dict(op=op, n_seqs=n, q=q, heads=rng.choice([16, 64]), kv=kv,
                 shared=rng.choice([0, _log(rng, 1, 65536), _log(rng, 1, 65536), 64 * _log(rng, 1, 1024)]), own_min=least,
                 own_max=least + _log(rng, 1, 4096))
        if work(c)["flops"] <= work(listed()[10])["flops"]:
            return c


# ------------------------------------------------------------------------------------------------ inputs
class Cache:
    """One layer's paged cache: kv [pages, 64, 576] bf16 or uint8 codes (or 656-byte rows), k_idx [pages, 64, d]."""

    def __init__(self, kv, kv_scale, k_idx, k_idx_scale, kv_dtype, idx_dtype):
        self.kv, self.kv_scale, self.k_idx, self.k_idx_scale = kv, kv_scale, k_idx, k_idx_scale
        self.kv_dtype, self.idx_dtype = kv_dtype, idx_dtype


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rope_table():
    """[MAX_POS][64] fp32: cos of 32 angles, then their sin; the angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    a = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _empty_cache(pages, kv, idx):
    d = IDX_D if idx == "fp8" else IDX_D // 2
    z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    rows = {"bf16": (D_QK, torch.bfloat16), "fp8": (D_QK, torch.uint8), "fp8_ds_mla": (DS_BYTES, torch.uint8)}[kv]
    return Cache(z(pages, PAGE, rows[0], dtype=rows[1]), z(pages, PAGE, dtype=torch.float32) if kv == "fp8" else None,
                 z(pages, PAGE, d, dtype=torch.uint8 if idx == "fp8" else torch.bfloat16),
                 z(pages, PAGE, dtype=torch.float32) if idx == "fp8" else None, kv, idx)


def _random_kv(g, pages, kv):
    """A filled latent pool: N(0,1) rows rounded to the format (scale = amax / 448)."""
    c = _empty_cache(pages, kv, "bf16")
    step = 4096
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), PAGE, D_QK, generator=g, device="cuda")
        b = a + x.shape[0]
        if kv == "bf16":
            c.kv[a:b] = x.to(torch.bfloat16)
        elif kv == "fp8":
            s = x.abs().amax(-1) / 448.0
            c.kv[a:b] = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c.kv_scale[a:b] = s
        else:
            t = x[..., :D_V].reshape(b - a, PAGE, 4, 128)
            s = t.abs().amax(-1) / 448.0
            c.kv[a:b, :, :D_V] = (t / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(b - a, PAGE, D_V)
            c.kv[a:b, :, D_V:D_V + 16] = s.contiguous().view(torch.uint8)
            c.kv[a:b, :, D_V + 16:] = x[..., D_V:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return c


def prepare(case, seed):
    g = _generator(seed)
    ints = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "tables":
        n = case["n_seqs"]
        s["ctx"], s["new"] = ints(case["ctx_min"], case["ctx_max"], n), ints(case["new_min"], case["new_max"], n)
        s["max_pages"] = -(-(case["ctx_max"] + case["new_max"]) // PAGE)
        s["max_new"] = max(1, n * case["new_max"])
        n_free = n * (-(-case["new_max"] // PAGE) + 1)
        held = (s["ctx"] + PAGE - 1) // PAGE
        perm = torch.randperm(n * s["max_pages"] + n_free, generator=g, device="cuda").to(torch.int32)
        s["free"] = perm[:n_free].contiguous()
        col = torch.arange(s["max_pages"], device="cuda")
        s["tables"] = torch.where(col[None] < held[:, None], perm[n_free:].view(n, -1), -1).contiguous()
        i = lambda k: new(k, dtype=torch.int32)  # noqa: E731
        s["out"] = dict(seq_lens=i(n), cu_new=i(n + 1), positions=i(s["max_new"]), slots=i(s["max_new"]), row_seq=i(s["max_new"]),
                        pages_used=i(1))
    elif case["op"] == "append":
        n = case["rows"]
        pages = -(-n // PAGE) + 3
        s["cache"] = _empty_cache(pages, case["kv"], case["idx"])
        d = s["cache"].k_idx.shape[-1]
        s["slots"] = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n].to(torch.int32)
        if case["holes"]:
            s["slots"][torch.rand(n, generator=g, device="cuda") < 0.1] = -1
        s["positions"] = ints(0, MAX_POS - 1, n)
        s["ckv"], s["k_raw"] = _normal(g, n, D_QK, std=1.7), _normal(g, n, d, std=1.3)
        s["kv_norm"] = 1 + 0.1 * _normal(g, D_V, dtype=torch.float32)
        s["idx_norm"], s["idx_bias"] = 1 + 0.1 * _normal(g, d, dtype=torch.float32), 0.1 * _normal(g, d, dtype=torch.float32)
        s["rope"] = _rope_table()
    elif case["op"] == "query":
        n, h = case["rows"], case["heads"]
        s["q"] = _normal(g, n, h, D_QK)  # the latent part is there already; the call fills the last 64 values
        s["q_proj"] = _normal(g, n, h, 192)  # each head's projection; its last 64 values are rotated
        s["q_raw"] = _normal(g, n, IDX_H, IDX_D, std=1.3)
        s["w"] = torch.rand(n, IDX_H, generator=g, device="cuda") + 0.1
        s["idx_norm"] = 1 + 0.1 * _normal(g, IDX_D, dtype=torch.float32)
        s["positions"] = ints(0, MAX_POS - 1, n)
        s["rope"] = _rope_table()
        s["q_idx"], s["w_out"] = new(n, IDX_H, IDX_D, dtype=torch.uint8), new(n, IDX_H, dtype=torch.float32)
    else:
        n, h, q, shared = case["n_seqs"], case["heads"], case["q"], case["shared"]
        s["seq_lens"] = shared + ints(case["own_min"], case["own_max"], n)
        s["max_seq_len"] = shared + case["own_max"]
        whole = shared // PAGE
        mine = -(-s["max_seq_len"] // PAGE) - whole
        pages = whole + n * mine
        s["cache"] = c = _random_kv(g, pages, case["kv"])
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["tables"] = torch.cat([perm[:whole].expand(n, whole), perm[whole:].view(n, mine)], 1).contiguous()
        if shared % PAGE:  # the shared prompt's last tokens lie in a page of each request's own, alike in all
            at, part = s["tables"][:, whole].long(), shared % PAGE
            c.kv[at, :part] = c.kv[at[0], :part].clone()
            if c.kv_scale is not None:
                c.kv_scale[at, :part] = c.kv_scale[at[0], :part].clone()
        s["q_rows"] = _normal(g, n * q, h, D_QK)
        s["sm_scale"] = 1.0 / math.sqrt(D_QK)
        s["out"], s["lse"] = new(n * q, h, D_V, dtype=torch.bfloat16), new(n * q, h, dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def _held(cache):
    """What the cache holds, 8-bit codes as the values that they stand for."""
    f8 = torch.float8_e4m3fn
    if cache.kv_dtype == "fp8_ds_mla":
        got = [cache.kv[..., :D_V].view(f8), cache.kv[..., D_V:D_V + 16].view(torch.float32), cache.kv[..., D_V + 16:].view(torch.bfloat16)]
    else:
        got = [cache.kv if cache.kv_dtype == "bf16" else cache.kv.view(f8)]
    if cache.kv_scale is not None:
        got.append(cache.kv_scale)
    got.append(cache.k_idx if cache.idx_dtype == "bf16" else cache.k_idx.view(f8))
    if cache.k_idx_scale is not None:
        got.append(cache.k_idx_scale)
    return got


def run(s):
    if own:
        return _run_own(s)
    return {"tables": _tables, "append": _append, "query": _query, "attention": _attention}[s["op"]](s)


def _run_own(s):
    import indexer_top_sparse_score_gb300 as smla
    if s["op"] == "tables":
        o = s["out"]
        s["ws"] = smla.build_tables(s["ctx"], s["new"], s["tables"], s["free"], s["max_new"], ws=s.get("ws"), **o)[-1]
        return [s["tables"], o]
    if s["op"] == "append":
        c = s["cache"]
        s["ws"] = smla.cache_append(c, s["slots"], s["positions"], s["rope"], ckv=s["ckv"], kv_norm=s["kv_norm"], k_idx=s["k_raw"],
                                    idx_norm=s["idx_norm"], idx_bias=s["idx_bias"], eps=EPS, ws=s.get("ws"))
        return _held(c)
    if s["op"] == "query":
        s["ws"] = smla.query_prep(s["positions"], s["rope"], q_pe=s["q_proj"][..., 128:], q=s["q"], q_idx_raw=s["q_raw"], w=s["w"],
                                  idx_dtype="fp8", idx_norm=s["idx_norm"], eps=EPS, w_scale=IDX_D ** -0.5, q_idx=s["q_idx"],
                                  w_out=s["w_out"], ws=s.get("ws"))[-1]
        return [s["q"], s["q_idx"].view(torch.float8_e4m3fn), s["w_out"]]
    _, _, s["ws"] = smla.shared_prefix_fwd(s["cache"], s["tables"], s["seq_lens"], s["max_seq_len"], s["shared"], s["q"], s["q_rows"],
                                           s["sm_scale"], out=s["out"], lse=s["lse"], ws=s.get("ws"))
    return [s["out"], s["lse"]]


def _tables(s):
    ctx, add, tables, free = s["ctx"], s["new"], s["tables"], s["free"]
    n, max_pages, max_new = ctx.shape[0], s["max_pages"], s["max_new"]
    held = (ctx + PAGE - 1) // PAGE
    need = (ctx + add + PAGE - 1) // PAGE - held
    first = need.cumsum(0) - need
    given = torch.minimum(need, (free.shape[0] - first).clamp_min(0))
    got = torch.minimum(add, (held + given) * PAGE - ctx)
    cu = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0).to(torch.int32)])
    col = torch.arange(max_pages, device="cuda")[None]
    fresh = (col >= held[:, None]) & (col < (held + given)[:, None])
    at = (first[:, None] + col - held[:, None]).clamp(0, free.shape[0] - 1)
    tables.copy_(torch.where(fresh, free[at], tables))
    i = torch.arange(max_new, device="cuda")
    b = torch.searchsorted(cu[1:], i.to(torch.int32), right=True).clamp_max(n - 1)
    k = i - cu[b]
    live = i < cu[n]
    pos = ctx[b] + k
    page = tables[b, (pos // PAGE).clamp_max(max_pages - 1)]
    o = s["out"]
    o["seq_lens"].copy_(ctx + got)
    o["cu_new"].copy_(cu)
    o["positions"].copy_(torch.where(live, pos, -1))
    o["row_seq"].copy_(torch.where(live, b, -1))
    o["slots"].copy_(torch.where(live & (k < got[b]), page * PAGE + pos % PAGE, -1))
    o["pages_used"].copy_(need.sum().clamp_max(free.shape[0]))
    return [tables, o]


def _rotate(x, cs, interleaved):
    """The 64 values of the last axis as 32 pairs, turned by the angles whose cos and sin `cs` holds."""
    c, d = cs[..., :32], cs[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * d, a * d + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * d, a * d + b * c], -1)


def _codes(x, shape=None):
    """(e4m3 codes as bytes, scale) of the values along the last axis: scale = largest magnitude / 448, 1 where all are zero."""
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, 1.0)
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _append(s):
    c, slots = s["cache"], s["slots"]
    live = slots >= 0
    at = slots[live].long()
    cs = s["rope"][s["positions"][live].long()]
    x = s["ckv"][live].float()
    lat = x[:, :D_V] * torch.rsqrt(x[:, :D_V].square().mean(-1, keepdim=True) + EPS) * s["kv_norm"]
    row = torch.cat([lat, _rotate(x[:, D_V:], cs, True)], 1)
    kv = c.kv.view(-1, c.kv.shape[-1])
    if c.kv_dtype == "bf16":
        kv[at] = row.to(torch.bfloat16)
    elif c.kv_dtype == "fp8":
        kv[at], c.kv_scale.view(-1)[at] = _codes(row)
    else:
        codes, scale = _codes(row[:, :D_V].reshape(-1, 4, 128))
        kv[at] = torch.cat([codes.reshape(-1, D_V), scale.contiguous().view(torch.uint8), row[:, D_V:].to(torch.bfloat16).view(torch.uint8)], 1)
    k = s["k_raw"][live].float()
    k = k - k.mean(-1, keepdim=True)
    k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["idx_norm"] + s["idx_bias"]
    k = torch.cat([_rotate(k[:, :ROPE], cs, False), k[:, ROPE:]], 1)
    ki = c.k_idx.view(-1, c.k_idx.shape[-1])
    if c.idx_dtype == "bf16":
        ki[at] = k.to(torch.bfloat16)
    else:
        ki[at], c.k_idx_scale.view(-1)[at] = _codes(k)
    return _held(c)


def _query(s):
    cs = s["rope"][s["positions"].long()][:, None]
    s["q"][..., D_V:] = _rotate(s["q_proj"][..., 128:].float(), cs, True).to(torch.bfloat16)
    x = s["q_raw"].float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["idx_norm"]
    codes, scale = _codes(torch.cat([_rotate(x[..., :ROPE], cs, False), x[..., ROPE:]], -1))
    s["q_idx"].copy_(codes)
    s["w_out"].copy_(s["w"] * (scale * IDX_D ** -0.5))
    return [s["q"], s["q_idx"].view(torch.float8_e4m3fn), s["w_out"]]


def _values(c, at, dtype=torch.float32):
    """The latent rows of pool rows `at` as numbers of `dtype`."""
    r = c.kv.view(-1, c.kv.shape[-1])[at]
    if c.kv_dtype == "bf16":
        return r.to(dtype)
    f8 = lambda v: v.view(torch.float8_e4m3fn).to(dtype)  # noqa: E731
    if c.kv_dtype == "fp8":
        return f8(r) * c.kv_scale.view(-1)[at][..., None].to(dtype)
    lat = f8(r[..., :D_V].contiguous()).unflatten(-1, (4, 128)) * r[..., D_V:D_V + 16].contiguous().view(torch.float32)[..., None].to(dtype)
    return torch.cat([lat.flatten(-2), r[..., D_V + 16:].contiguous().view(torch.bfloat16).to(dtype)], -1)


def _attention(s):
    c, tables, n, q, h, shared = s["cache"], s["tables"].long(), s["n_seqs"], s["q"], s["heads"], s["shared"]
    place = lambda t, p: t[..., p // PAGE] * PAGE + p % PAGE  # noqa: E731
    ps, po = torch.arange(shared, device="cuda"), torch.arange(shared, s["max_seq_len"], device="cuda")
    pos = s["seq_lens"][:, None] - q + torch.arange(q, device="cuda")  # [n, q]
    x = s["q_rows"].float() * s["sm_scale"]
    ks, ko = _values(c, place(tables[0], ps)), _values(c, place(tables, po))
    ss = (x.view(n * q * h, D_QK) @ ks.T).view(n, q, h, shared).masked_fill_((ps > pos[..., None])[:, :, None], -math.inf)
    so = torch.bmm(x.view(n, q * h, D_QK), ko.mT).view(n, q, h, -1).masked_fill_((po > pos[..., None])[:, :, None], -math.inf)
    m = torch.maximum(ss.amax(-1), so.amax(-1)) if shared else so.amax(-1)
    z = torch.where(m == -math.inf, 0.0, m)[..., None]
    ss, so = ss.sub_(z).exp_(), so.sub_(z).exp_()
    l = ss.sum(-1) + so.sum(-1)
    o = (ss.view(n * q * h, shared) @ ks[:, :D_V]).view(n, q, h, D_V) + torch.bmm(so.view(n, q * h, -1), ko[..., :D_V]).view(n, q, h, D_V)
    s["out"].copy_((o / torch.where(l > 0, l, 1.0)[..., None]).view(n * q, h, D_V))
    s["lse"].copy_((z[..., 0] + l.log()).view(n * q, h))
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
_ROW = {"bf16": 2 * D_QK, "fp8": D_QK + 4, "fp8_ds_mla": DS_BYTES}


def work(case):
    if case["op"] == "tables":
        n, tokens = case["n_seqs"], case["n_seqs"] * (case["new_min"] + case["new_max"]) / 2
        return {"bytes": 16.0 * n + 12.0 * max(1, n * case["new_max"]) + 8.0 * (tokens / PAGE + n / 2), "flops": 0.0}
    if case["op"] == "append":
        n = case["rows"]
        idx = IDX_D + 4 if case["idx"] == "fp8" else IDX_D
        raw = 2 * D_QK + (2 * IDX_D if case["idx"] == "fp8" else IDX_D)
        return {"bytes": float(n) * (raw + _ROW[case["kv"]] + idx + 8 + 4 * ROPE), "flops": 12.0 * n * (D_QK + IDX_D)}
    if case["op"] == "query":
        n, h = case["rows"], case["heads"]
        return {"bytes": float(n) * (h * ROPE * 4 + IDX_H * (3 * IDX_D + 8) + 4 + 4 * ROPE), "flops": n * (6.0 * h * ROPE + 12.0 * IDX_H * IDX_D)}
    n, q, h = case["n_seqs"], case["q"], case["heads"]
    mine = (case["own_min"] + case["own_max"]) / 2
    seen = case["shared"] + mine - (q - 1) / 2  # keys of a middle new token
    return {"bytes": (case["shared"] + n * mine) * _ROW[case["kv"]] + n * q * h * (2 * D_QK + 2 * D_V + 4.0),
            "flops": 2.0 * n * q * h * seen * (D_QK + D_V)}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "tables":
        return None
    if case["op"] == "attention":
        return _exact_attention(case, s)
    angle = lambda p: torch.polar(torch.ones((), dtype=f, device="cuda"), p)  # noqa: E731
    inv = torch.exp(torch.arange(32, dtype=f, device="cuda") * (-math.log(10000.0) / 32))
    turn = angle(s["positions"].to(f)[:, None] * inv)  # complex: one turn a pair

    def pairs(x, t):  # neighbours are a pair
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous()) * t
        return torch.view_as_real(z).reshape(x.shape)

    def halves(x, t):  # value i and value i + 32 are a pair
        z = torch.complex(x[..., :32].contiguous(), x[..., 32:64].contiguous()) * t
        return torch.cat([z.real, z.imag, x[..., 64:]], -1)

    def scale(x):
        top = x.abs().max(-1).values / 448
        return torch.where(top == 0, torch.ones_like(top), top)

    def codes(x):
        return (x / scale(x)[..., None]).float().to(torch.float8_e4m3fn).to(f)

    if case["op"] == "append":
        c, live = s["cache"], s["slots"] >= 0
        at = s["slots"][live].long()

        def pool(like, v):
            out = torch.zeros(like.shape[0] * PAGE, *v.shape[1:], dtype=f, device="cuda")
            out[at] = v[live]
            return out.view(like.shape[0], PAGE, *v.shape[1:])

        x = s["ckv"].to(f)
        lat = x[:, :D_V] / torch.sqrt((x[:, :D_V] ** 2).sum(-1, keepdim=True) / D_V + EPS) * s["kv_norm"].to(f)
        pe = pairs(x[:, D_V:], turn)
        row = torch.cat([lat, pe], -1)
        if case["kv"] == "bf16":
            got = [pool(c.kv, row)]
        elif case["kv"] == "fp8":
            got = [pool(c.kv, codes(row)), pool(c.kv, scale(row))]
        else:
            t = lat.view(-1, 4, 128)
            got = [pool(c.kv, codes(t).view(-1, D_V)), pool(c.kv, scale(t)), pool(c.kv, pe)]
        k = s["k_raw"].to(f)
        var, mean = torch.var_mean(k, -1, correction=0, keepdim=True)
        k = halves((k - mean) / torch.sqrt(var + EPS) * s["idx_norm"].to(f) + s["idx_bias"].to(f), turn)
        return got + ([pool(c.kv, k)] if case["idx"] == "bf16" else [pool(c.kv, codes(k)), pool(c.kv, scale(k))])
    q = s["q"].to(f)
    q[..., D_V:] = pairs(s["q_proj"][..., 128:].to(f), turn[:, None])
    x = s["q_raw"].to(f)
    x = halves(x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / IDX_D + EPS) * s["idx_norm"].to(f), turn[:, None])
    return [q, codes(x), s["w"].to(f) * scale(x) / math.sqrt(IDX_D)]


def _exact_attention(case, s):
    """Each request alone, through its own table: softmax over all of its keys, a few tokens at a time."""
    f, q, h, c = torch.float64, case["q"], case["heads"], s["cache"]
    out = torch.zeros(case["n_seqs"] * q, h, D_V, dtype=f, device="cuda")
    lse = torch.full((case["n_seqs"] * q, h), -math.inf, dtype=f, device="cuda")
    for b, length in enumerate(s["seq_lens"].tolist()):
        p = torch.arange(length, device="cuda")
        k = _values(c, s["tables"][b].long()[p // PAGE] * PAGE + p % PAGE, f)
        for j in range(0, q, 32):
            e = min(q, j + 32)
            x = s["q_rows"][b * q + j:b * q + e].to(f)
            z = torch.einsum("thd,sd->ths", x, k) * s["sm_scale"]
            z = torch.where(p <= torch.arange(length - q + j, length - q + e, device="cuda")[:, None, None], z, -math.inf)
            lse[b * q + j:b * q + e] = torch.logsumexp(z, -1)
            out[b * q + j:b * q + e] = torch.einsum("ths,sd->thd", torch.softmax(z, -1), k[:, :D_V])
    return [out, lse]
