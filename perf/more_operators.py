"""Measured cases of the operators that compute prompts in the expanded form of latent attention.

Where a prompt is dense (its keys are not selected), a model turns the cached latent rows into keys and values of
each head and attends over those. Around that product of its own it calls:
  table   the rotation table of a range of positions, plain or scaled for long contexts;
  rope    rotation of a part of each head of queries or keys;
  read    rows of the paged cache back as bf16 values: latent part, rope part, indexer keys;
  prompt  attention over packed prompts with grouped heads, the keys' rope part shared by all heads, joined with the
          result over another part of the keys.
`run` computes them with elementary torch operations (own = False) or through the package (own = True).
"""
import math

import torch

own = False

PAGE, D_QK, D_LAT, ROPE, D_V = 64, 576, 512, 64, 128
IDX_D, DS_BYTES = 128, 656
MAX_POS = 1 << 17


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the table of a model of 8K positions, and one of a million with a ramped scaling by 32
        dict(name="table 8K", op="table", n=8192, first=0, dim=64, base=10000.0, factor=1.0, original=0),
        dict(name="table 1M ramped", op="table", n=1048576, first=0, dim=64, base=10000.0, factor=32.0, original=32768),
        # the queries of the decode batch (64 requests, 2 tokens), and of one prefill chunk, half-split pairs
        dict(name="rope 128x64", op="rope", rows=128, heads=64, width=192, dim=64, interleaved=True),
        dict(name="rope 8192x64 halves", op="rope", rows=8192, heads=64, width=192, dim=64, interleaved=False),
        # a few hundred cached tokens of one request; the whole cache of a ragged batch; a 131,072-token request
        dict(name="read ds_mla 1x600", op="read", n_seqs=1, len_min=600, len_max=600, kv="fp8_ds_mla", keys=False),
        dict(name="read bf16 37 ragged", op="read", n_seqs=37, len_min=1, len_max=2047, kv="bf16", keys=True),
        dict(name="read fp8 1x131072", op="read", n_seqs=1, len_min=131072, len_max=131072, kv="fp8", keys=False),
        # the smallest prompt call: one short prompt of 16 heads
        dict(name="prompt 1x100 h16", op="prompt", n_seqs=1, q_min=100, q_max=100, ctx_min=0, ctx_max=0, heads=16, kv_heads=16, dim=192,
             pe=True, causal=True, join=False),
        # a ragged batch of prompts that are all within the top-k
        dict(name="prompt 37 ragged 2K", op="prompt", n_seqs=37, q_min=1, q_max=2047, ctx_min=0, ctx_max=0, heads=64, kv_heads=64, dim=192,
             pe=True, causal=True, join=False),
        # grouped heads without a rope part of their own: 64 heads on 8, 8,192 tokens
        dict(name="prompt 1x8192 64 on 8", op="prompt", n_seqs=1, q_min=8192, q_max=8192, ctx_min=0, ctx_max=0, heads=64, kv_heads=8, dim=128,
             pe=False, causal=True, join=False),
        # few new tokens of several requests against a part of their contexts, joined with the part before
        dict(name="prompt 5x3 on 9K joined", op="prompt", n_seqs=5, q_min=3, q_max=3, ctx_min=8001, ctx_max=9999, heads=64, kv_heads=64,
             dim=192, pe=True, causal=False, join=True),
        # the largest: a 16,384-token prompt
        dict(name="prompt 1x16384", op="prompt", n_seqs=1, q_min=16384, q_max=16384, ctx_min=0, ctx_max=0, heads=64, kv_heads=64, dim=192,
             pe=True, causal=True, join=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "read", "prompt", "prompt", "prompt"])
    if op == "table":
        scaled = rng.choice([0, 1, 2])  # plain, linear, ramped
        return dict(op=op, n=_log(rng, 1, 1 << 20), first=rng.choice([0, _log(rng, 1, 1 << 20)]), dim=rng.choice([32, 64, 64, 128]),
                    base=rng.choice([10000.0, 1e6]), factor=1.0 if scaled == 0 else round(rng.uniform(1.5, 40.0), 2),
                    original=rng.choice([4096, 32768]) if scaled == 2 else 0)
    if op == "rope":
        dim = rng.choice([32, 64, 64, 128])
        return dict(op=op, rows=_log(rng, 1, 8192), heads=rng.choice([1, 8, 16, 64]), width=dim + rng.choice([0, 64, 128]), dim=dim,
                    interleaved=rng.random() < 0.5)
    if op == "read":
        n = _log(rng, 1, 300)
        return dict(op=op, n_seqs=n, len_min=rng.choice([0, 1]), len_max=_log(rng, 1, 131072 // n), kv=rng.choice(["bf16", "fp8", "fp8_ds_mla"]),
                    keys=rng.random() < 0.5)
    while True:
        n = rng.choice([1, _log(rng, 1, 64)])
        causal = rng.random() < 0.75
        ctx = rng.choice([0, 0, _log(rng, 1, 16384)]) if causal else _log(rng, 1, 16384)
        heads, kv_heads = rng.choice([(16, 16), (64, 64), (64, 64), (64, 8), (64, 1), (12, 4)])
        dim, pe = rng.choice([(192, True), (192, True), (192, False), (128, False)])
        q = rng.choice([_log(rng, 1, 16384 // n), _log(rng, 1, 16384 // n), _log(rng, 1, 8)])
        c = dict(op=op, n_seqs=n, q_min=rng.choice([1, q]), q_max=q, ctx_min=ctx // 2, ctx_max=ctx, heads=heads, kv_heads=kv_heads, dim=dim,
                 pe=pe, causal=causal, join=rng.random() < 0.4)
        if work(c)["flops"] <= work(listed()[11])["flops"] and c["n_seqs"] * (ctx + q) * kv_heads <= 32768 * 64:
            return c


# ------------------------------------------------------------------------------------------------ inputs
class Cache:
    """One layer's paged cache: kv [pages, 64, 576] bf16 or uint8 codes (or 656-byte rows), k_idx [pages, 64, 128]."""

    def __init__(self, kv, kv_scale, k_idx, k_idx_scale, kv_dtype, idx_dtype):
        self.kv, self.kv_scale, self.k_idx, self.k_idx_scale = kv, kv_scale, k_idx, k_idx_scale
        self.kv_dtype, self.idx_dtype = kv_dtype, idx_dtype


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _codes(x):
    """(e4m3 codes as bytes, scale) of the values along the last axis."""
    s = x.abs().amax(-1) / 448.0
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _filled_cache(g, pages, kv):
    """A filled pool: N(0,1) rows and indexer keys rounded to the format (scale = amax / 448)."""
    z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    width, dtype = {"bf16": (D_QK, torch.bfloat16), "fp8": (D_QK, torch.uint8), "fp8_ds_mla": (DS_BYTES, torch.uint8)}[kv]
    c = Cache(z(pages, PAGE, width, dtype=dtype), z(pages, PAGE, dtype=torch.float32) if kv == "fp8" else None,
              z(pages, PAGE, IDX_D, dtype=torch.uint8), z(pages, PAGE, dtype=torch.float32), kv, "fp8")
    for a in range(0, pages, 4096):
        b = min(pages, a + 4096)
        x = torch.randn(b - a, PAGE, D_QK, generator=g, device="cuda")
        if kv == "bf16":
            c.kv[a:b] = x.to(torch.bfloat16)
        elif kv == "fp8":
            c.kv[a:b], c.kv_scale[a:b] = _codes(x)
        else:
            codes, s = _codes(x[..., :D_LAT].reshape(b - a, PAGE, 4, 128))
            c.kv[a:b, :, :D_LAT] = codes.reshape(b - a, PAGE, D_LAT)
            c.kv[a:b, :, D_LAT:D_LAT + 16] = s.contiguous().view(torch.uint8)
            c.kv[a:b, :, D_LAT + 16:] = x[..., D_LAT:].to(torch.bfloat16).contiguous().view(torch.uint8)
        c.k_idx[a:b], c.k_idx_scale[a:b] = _codes(torch.randn(b - a, PAGE, IDX_D, generator=g, device="cuda"))
    return c


def _lengths(g, lo, hi, n):
    """n lengths of lo .. hi whose sum is the same for every seed: each has its counterpart lo + hi - length."""
    half = torch.randint(lo, hi + 1, (n // 2,), generator=g, device="cuda", dtype=torch.int32)
    middle = torch.full((n % 2,), (lo + hi) // 2, dtype=torch.int32, device="cuda")
    return torch.cat([half, middle, lo + hi - half])


def _cumulated(lens):
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    return cu


def prepare(case, seed):
    g = _generator(seed)
    ints = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "table":
        # a table of another seed begins at another position
        s["first"] = case["first"] + int(seed) % 1009
        s["out"] = new(case["n"], case["dim"], dtype=torch.float32)
    elif case["op"] == "rope":
        n, d = case["rows"], case["dim"]
        a = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        s["table"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        s["positions"] = ints(0, MAX_POS - 1, n)
        s["x"] = _normal(g, n, case["heads"], case["width"])[..., case["width"] - d:]  # the last values of each head
        s["out"] = new(n, case["heads"], d, dtype=torch.bfloat16)
    elif case["op"] == "read":
        n = case["n_seqs"]
        lens = _lengths(g, case["len_min"], case["len_max"], n)
        s["starts"] = torch.zeros_like(lens)  # the later part of what a request holds
        if case["len_max"] < 65536:
            s["starts"] = ints(0, 200, n)
        s["cu"] = _cumulated(lens)
        s["rows"] = int(s["cu"][-1])
        width = -(-int((lens + s["starts"]).max()) // PAGE) + 1
        pages = max(1, int(((lens + s["starts"] + PAGE - 1) // PAGE).sum()))
        s["cache"] = _filled_cache(g, pages, case["kv"])
        held = (lens + s["starts"] + PAGE - 1) // PAGE
        first = held.cumsum(0) - held
        col = torch.arange(width, device="cuda")[None]
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["tables"] = torch.where(col < held[:, None], perm[(first[:, None] + col).clamp_max(pages - 1)], -1).to(torch.int32).contiguous()
        rows = max(1, s["rows"])
        s["latent"], s["pe"] = new(rows, D_LAT, dtype=torch.bfloat16), new(rows, ROPE, dtype=torch.bfloat16)
        s["latent"].zero_(), s["pe"].zero_()
        s["keys_out"] = torch.zeros(rows, IDX_D, dtype=torch.bfloat16, device="cuda") if case["keys"] else None
    else:
        n, h, hk, d = case["n_seqs"], case["heads"], case["kv_heads"], case["dim"]
        ql, ctx = _lengths(g, case["q_min"], case["q_max"], n), _lengths(g, case["ctx_min"], case["ctx_max"], n)
        kl = ctx + ql if case["causal"] else ctx  # causal: the new tokens' own keys come last
        s["cu_q"], s["cu_k"] = _cumulated(ql), _cumulated(kl)
        s["ql"], s["kl"] = ql.tolist(), kl.tolist()
        tq, tk = sum(s["ql"]), max(1, sum(s["kl"]))
        own_d = d - ROPE if case["pe"] else d
        kv = _normal(g, tk, hk, own_d + D_V)  # the up-projection's result: a head's keys, then its values
        s["q"], s["k"], s["v"] = _normal(g, tq, h, d), kv[..., :own_d], kv[..., own_d:]
        s["k_pe"] = _normal(g, tk, ROPE) if case["pe"] else None
        s["sm_scale"] = 1.0 / math.sqrt(d)
        s["prev_out"] = s["prev_lse"] = None
        if case["join"]:
            s["prev_out"], s["prev_lse"] = _normal(g, tq, h, D_V, dtype=torch.float32), 6.0 + _normal(g, tq, h, dtype=torch.float32)
        s["out"], s["lse"] = new(tq, h, D_V, dtype=torch.bfloat16), new(tq, h, dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"table": _table, "rope": _rope, "read": _read, "prompt": _prompt}[s["op"]](s)


def _run_own(s):
    import indexer_top_sparse_score_gb300 as smla
    if s["op"] == "table":
        return [smla.rope_table(s["n"], s["dim"], first=s["first"], base=s["base"], factor=s["factor"], original=s["original"],
                                magnitude=_magnitude(s), out=s["out"])]
    if s["op"] == "rope":
        _, s["ws"] = smla.rope_apply(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], out=s["out"], ws=s.get("ws"))
        return [s["out"]]
    if s["op"] == "read":
        s["ws"] = smla.cache_read(s["cache"], s["tables"], s["cu"], max(1, s["rows"]), starts=s["starts"], latent=s["latent"], pe=s["pe"],
                                  keys=s["keys_out"], ws=s.get("ws"))[-1]
        return [s["latent"], s["pe"]] + ([s["keys_out"]] if s["keys"] else [])
    _, _, s["ws"] = smla.prompt_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["sm_scale"], k_pe=s["k_pe"], causal=s["causal"],
                                    prev_out=s["prev_out"], prev_lse=s["prev_lse"], out=s["out"], lse=s["lse"], ws=s.get("ws"))
    return [s["out"], s["lse"]]


def _magnitude(s):
    return 1.0 + 0.1 * math.log(s["factor"]) if s["original"] else 1.0


def _frequencies(s):
    """Turns in radians per position of each pair, in 64 bits."""
    dim, base, factor = s["dim"], s["base"], s["factor"]
    i = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    inv = base ** (-2.0 * i / dim)
    if not s["original"]:
        return inv / factor
    at = lambda beta: dim * math.log(s["original"] / (beta * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), dim - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return inv * (1.0 - ramp) + inv / factor * ramp


def _table(s):
    a = torch.arange(s["first"], s["first"] + s["n"], device="cuda", dtype=torch.float64)[:, None] * _frequencies(s)
    h = s["dim"] // 2
    s["out"][:, :h] = (a.cos() * _magnitude(s)).float()
    s["out"][:, h:] = (a.sin() * _magnitude(s)).float()
    return [s["out"]]


def _rope(s):
    h = s["dim"] // 2
    cs = s["table"][s["positions"].long()][:, None]
    c, d, x = cs[..., :h], cs[..., h:], s["x"].float()
    if s["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * c - b * d, a * d + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:]
        y = torch.cat([a * c - b * d, a * d + b * c], -1)
    s["out"].copy_(y)
    return [s["out"]]


def _pool_rows(s):
    """Pool row of each output row."""
    i = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:].contiguous(), i, right=True)
    pos = (s["starts"][b] + i - s["cu"][b]).long()
    return s["tables"][b, pos // PAGE].long() * PAGE + pos % PAGE


def _read(s):
    c, at, n = s["cache"], _pool_rows(s), s["rows"]
    f8 = lambda v: v.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    r = c.kv.view(-1, c.kv.shape[-1])[at]
    if c.kv_dtype == "bf16":
        x = r
    elif c.kv_dtype == "fp8":
        x = (f8(r) * c.kv_scale.view(-1)[at][:, None]).to(torch.bfloat16)
    else:
        lat = f8(r[:, :D_LAT]).view(-1, 4, 128) * r[:, D_LAT:D_LAT + 16].contiguous().view(torch.float32)[..., None]
        x = torch.cat([lat.view(-1, D_LAT).to(torch.bfloat16), r[:, D_LAT + 16:].contiguous().view(torch.bfloat16)], 1)
    s["latent"][:n] = x[:, :D_LAT]
    s["pe"][:n] = x[:, D_LAT:]
    if not s["keys"]:
        return [s["latent"], s["pe"]]
    s["keys_out"][:n] = (f8(c.k_idx.view(-1, IDX_D)[at]) * c.k_idx_scale.view(-1)[at][:, None]).to(torch.bfloat16)
    return [s["latent"], s["pe"], s["keys_out"]]


def _prompt(s):
    h, hk, d, dev = s["heads"], s["kv_heads"], s["dim"], "cuda"
    q0 = k0 = 0
    step = 1024
    for nq, nk in zip(s["ql"], s["kl"]):
        for a in range(0, nq, step):
            e = min(nq, a + step)
            end = min(nk, max(0, nk - nq + e)) if s["causal"] else nk  # keys that the last of these tokens sees
            per = max(1, min(hk, (1 << 28) // max(1, (e - a) * end * (h // hk))))
            pos = torch.arange(nk - nq + a, nk - nq + e, device=dev)
            for g in range(0, hk, per):
                f = min(hk, g + per)
                heads = slice(g * (h // hk), f * (h // hk))
                k = s["k"][k0:k0 + end, g:f].float()
                if s["pe"]:
                    k = torch.cat([k, s["k_pe"][k0:k0 + end, None].float().expand(-1, f - g, -1)], -1)
                k, v = k.transpose(0, 1)[:, None], s["v"][k0:k0 + end, g:f].float().transpose(0, 1)[:, None]
                q = (s["q"][q0 + a:q0 + e, heads].float() * s["sm_scale"]).transpose(0, 1).unflatten(0, (f - g, h // hk))
                z = q @ k.mT
                if s["causal"]:
                    z.masked_fill_(torch.arange(end, device=dev) > pos[:, None], -math.inf)
                m = z.amax(-1, keepdim=True) if end else torch.full((*z.shape[:-1], 1), -math.inf, device=dev)
                m = torch.where(m == -math.inf, 0.0, m)
                p = z.sub_(m).exp_()
                l = p.sum(-1, keepdim=True)
                o = (p @ v) / torch.where(l > 0, l, 1.0)
                lse = (m + l.log())[..., 0].flatten(0, 1).T
                o = o.flatten(0, 1).transpose(0, 1)
                if s["join"]:
                    was = s["prev_lse"][q0 + a:q0 + e, heads]
                    both = torch.logaddexp(was, lse)
                    o = (was - both).exp()[..., None] * s["prev_out"][q0 + a:q0 + e, heads] + (lse - both).exp()[..., None] * o
                    lse = both
                s["out"][q0 + a:q0 + e, heads] = o.to(torch.bfloat16)
                s["lse"][q0 + a:q0 + e, heads] = lse
        q0, k0 = q0 + nq, k0 + nk
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
_ROW = {"bf16": 2 * D_QK, "fp8": D_QK + 4, "fp8_ds_mla": DS_BYTES}


def work(case):
    if case["op"] == "table":
        return {"bytes": 4.0 * case["n"] * case["dim"], "flops": 0.0}
    if case["op"] == "rope":
        n, d = case["rows"], case["dim"]
        return {"bytes": float(n) * (4 * case["heads"] * d + 4 * d + 4), "flops": 3.0 * n * case["heads"] * d}
    if case["op"] == "read":
        n = case["n_seqs"] * (case["len_min"] + case["len_max"]) / 2
        return {"bytes": n * (_ROW[case["kv"]] + 2 * D_QK + (3 * IDX_D + 4 if case["keys"] else 0)), "flops": 0.0}
    n, h, hk, d = case["n_seqs"], case["heads"], case["kv_heads"], case["dim"]
    q, ctx = (case["q_min"] + case["q_max"]) / 2, (case["ctx_min"] + case["ctx_max"]) / 2
    q2 = q * q + ((case["q_max"] - case["q_min"] + 1) ** 2 - 1) / 12  # mean square of the lengths
    pairs = n * (q * ctx + (q2 + q) / 2 if case["causal"] else q * ctx)  # of a token and a key that it sees
    keys = n * (ctx + q if case["causal"] else ctx)
    own_d = d - ROPE if case["pe"] else d
    return {"bytes": n * q * h * (2 * d + 2 * D_V + 4.0 + (4 * D_V + 4 if case["join"] else 0)) + keys * 2.0 * (
        hk * (own_d + D_V) + (ROPE if case["pe"] else 0)), "flops": 2.0 * pairs * h * (d + D_V)}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "table":
        p = torch.arange(case["n"], device="cuda") + s["first"]
        z = torch.polar(torch.full((), _magnitude(case), dtype=f, device="cuda"), torch.outer(p.to(f), _exact_frequencies(case)))
        return [torch.cat([z.real, z.imag], 1)]
    if case["op"] == "rope":
        x, half = s["x"].to(f), case["dim"] // 2
        pair = (lambda t: t.unflatten(-1, (half, 2))) if case["interleaved"] else (lambda t: t.unflatten(-1, (2, half)).mT)
        # the table is an input: its values as they are
        z = torch.view_as_complex(pair(x).contiguous()) * torch.complex(*s["table"].to(f)[s["positions"].long()][:, None].split(half, -1))
        y = torch.view_as_real(z)
        return [(y if case["interleaved"] else y.mT).reshape(x.shape)]
    if case["op"] == "read":
        return _exact_read(s, f)
    if work(case)["flops"] > 2e13:
        return None
    return _exact_prompt(s, f)


def _exact_frequencies(case):
    dim, out = case["dim"], []
    for i in range(dim // 2):
        w = math.exp(-2.0 * i / dim * math.log(case["base"]))
        if case["original"]:
            edge = [dim / 2 * (math.log(case["original"]) - math.log(2 * math.pi * b)) / math.log(case["base"]) for b in (32.0, 1.0)]
            low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), dim - 1)
            part = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            w = w * (1.0 - part + part / case["factor"])
        else:
            w = w / case["factor"]
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_read(s, f):
    c = s["cache"]
    outs = [torch.zeros(max(1, s["rows"]), w, dtype=f, device="cuda") for w in (D_LAT, ROPE, IDX_D)]
    for b, (lo, hi, start) in enumerate(zip(s["cu"].tolist()[:-1], s["cu"].tolist()[1:], s["starts"].tolist())):
        if hi == lo:
            continue
        first, last = start // PAGE, (start + hi - lo - 1) // PAGE
        ids, cut = s["tables"][b, first:last + 1].long(), slice(start - first * PAGE, start - first * PAGE + hi - lo)
        rows = c.kv[ids].flatten(0, 1)[cut]
        if c.kv_dtype == "bf16":
            x = rows.to(f)
        elif c.kv_dtype == "fp8":
            x = rows.view(torch.float8_e4m3fn).to(f) * c.kv_scale[ids].flatten()[cut, None].to(f)
        else:
            scale = rows[:, D_LAT:D_LAT + 16].contiguous().view(torch.float32).to(f).repeat_interleave(128, 1)
            x = torch.cat([rows[:, :D_LAT].contiguous().view(torch.float8_e4m3fn).to(f) * scale,
                           rows[:, D_LAT + 16:].contiguous().view(torch.bfloat16).to(f)], 1)
        outs[0][lo:hi], outs[1][lo:hi] = x[:, :D_LAT], x[:, D_LAT:]
        outs[2][lo:hi] = c.k_idx[ids].flatten(0, 1)[cut].view(torch.float8_e4m3fn).to(f) * c.k_idx_scale[ids].flatten()[cut, None].to(f)
    return outs if s["keys"] else outs[:2]


def _exact_prompt(s, f):
    """Each request and head alone, softmax over the keys that a token sees, some hundred tokens at a time."""
    h, group = s["heads"], s["heads"] // s["kv_heads"]
    out, lse = torch.zeros_like(s["out"], dtype=f), torch.full_like(s["lse"], -math.inf, dtype=f)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(s["n_seqs"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if nq == 0 or nk == 0:
            continue
        pe = s["k_pe"][ck[b]:ck[b + 1]].to(f) if s["pe"] else None
        for j in range(0, nq, 512):
            e = min(nq, j + 512)
            last = min(nk, nk - nq + e) if s["causal"] else nk
            if last <= 0:
                continue
            seen = torch.arange(last, device="cuda")[None] <= (
                torch.arange(j, e, device="cuda")[:, None] + (nk - nq) if s["causal"] else nk)
            per = max(1, (1 << 27) // ((e - j) * last * group))
            for g in range(0, s["kv_heads"], per):
                n = min(per, s["kv_heads"] - g)
                k = s["k"][ck[b]:ck[b] + last, g:g + n].to(f)
                x = s["q"][cq[b] + j:cq[b] + e, g * group:(g + n) * group].to(f).unflatten(1, (n, group))
                z = torch.einsum("tgrd,sgd->grts", x[..., :k.shape[-1]], k)
                if pe is not None:
                    z = z + torch.einsum("tgrd,sd->grts", x[..., k.shape[-1]:], pe[:last])
                z = torch.where(seen, z * s["sm_scale"], -math.inf)
                w = torch.softmax(z, -1) if last else z
                v = s["v"][ck[b]:ck[b] + last, g:g + n].to(f)
                o = torch.einsum("grts,sgd->tgrd", w, v).flatten(1, 2)
                at = (slice(cq[b] + j, cq[b] + e), slice(g * group, (g + n) * group))
                out[at] = torch.where(seen.any(-1)[:, None, None], o, 0.0)
                lse[at] = torch.logsumexp(z, -1).flatten(0, 1).T
    if s["join"]:
        was = s["prev_lse"].to(f)
        share = torch.sigmoid(lse - was)[..., None]  # of the part computed here
        out = share * out + (1 - share) * s["prev_out"].to(f)
        lse = torch.logsumexp(torch.stack([lse, was]), 0)
    return [out, lse]
