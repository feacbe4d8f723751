"""Inputs and 64-bit references of the serving operators' tests (plain numpy and
torch on the CPU, written from the formulas; nothing of the package's kernels)."""
import math

import numpy as np
import torch

PAGE, D_QK, D_V = 64, 576, 512


class Cache:
    """A paged cache by its tensors (what the package's entry points take)."""

    def __init__(self, kv, kv_scale, k_idx, k_idx_scale, kv_dtype, idx_dtype):
        self.kv, self.kv_scale, self.k_idx, self.k_idx_scale = kv, kv_scale, k_idx, k_idx_scale
        self.kv_dtype, self.idx_dtype = kv_dtype, idx_dtype

    def to(self, dev):
        f = lambda t: None if t is None else t.to(dev)  # noqa: E731
        return Cache(f(self.kv), f(self.kv_scale), f(self.k_idx), f(self.k_idx_scale), self.kv_dtype, self.idx_dtype)


def empty_cache(pages, kv_dtype="bf16", idx_dtype="fp8", fill=0, key_scale=True):
    """A cache whose bytes are all `fill`."""
    width = {"bf16": 2 * D_QK, "fp8": D_QK, "fp8_ds_mla": 656}[kv_dtype]
    kv = torch.full((pages, PAGE, width), fill, dtype=torch.uint8)
    ki = torch.full((pages, PAGE, 128), fill, dtype=torch.uint8)
    return Cache(kv.view(torch.bfloat16) if kv_dtype == "bf16" else kv,
                 torch.zeros(pages, PAGE) if kv_dtype == "fp8" else None,
                 ki.view(torch.bfloat16) if idx_dtype == "bf16" else ki,
                 torch.zeros(pages, PAGE) if idx_dtype == "fp8" and key_scale else None, kv_dtype, idx_dtype)


def filled_cache(pages, kv_dtype, seed, std=1.0):
    """Latent rows N(0, std) in the cache's format."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(pages, PAGE, D_QK, generator=g) * std
    c = empty_cache(pages, kv_dtype)
    if kv_dtype == "bf16":
        c.kv = x.to(torch.bfloat16)
    elif kv_dtype == "fp8":
        s = x.abs().amax(-1) / 448
        c.kv = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c.kv_scale = s
    else:
        t = x[..., :D_V].reshape(pages, PAGE, 4, 128)
        s = t.abs().amax(-1) / 448
        c.kv[..., :D_V] = (t / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(2)
        c.kv[..., D_V:D_V + 16] = s.contiguous().view(torch.uint8)
        c.kv[..., D_V + 16:] = x[..., D_V:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return c


def latent_values(c):
    """[pages * 64, 576] float64: what the latent rows hold."""
    n = c.kv.shape[0] * PAGE
    f8 = lambda b: b.contiguous().view(torch.float8_e4m3fn).float().double().numpy()  # noqa: E731
    kv = c.kv.cpu().reshape(n, -1)
    if c.kv_dtype == "bf16":
        return kv.float().double().numpy()
    if c.kv_dtype == "fp8":
        return f8(kv) * c.kv_scale.cpu().double().numpy().reshape(n, 1)
    s = kv[:, D_V:D_V + 16].contiguous().view(torch.float32).double().numpy()
    lat = f8(kv[:, :D_V]) * np.repeat(s, 128, axis=1)
    return np.concatenate([lat, kv[:, D_V + 16:].contiguous().view(torch.bfloat16).float().double().numpy()], 1)


# ---------------------------------------------------------------------------- tables
def tables_reference(ctx, new, tables, free, max_new):
    """smla_build_tables, one request and one token at a time."""
    n, max_pages = tables.shape
    tables = tables.copy()
    seq, cu = np.zeros(n, np.int32), np.zeros(n + 1, np.int32)
    pos, slot, own = (np.full(max_new, -1, np.int32) for _ in range(3))
    row, taken, wanted, bad = 0, 0, 0, False
    for b in range(n):
        c, a = int(ctx[b]), int(new[b])
        cu[b] = row
        if c < 0 or a < 0 or c + a > max_pages * PAGE:
            bad, c, a = True, 0, 0
        if a > max_new - row:
            bad, a = True, max_new - row
        seq[b] = c
        held = -(-c // PAGE)
        for k in range(a):
            t = c + k
            if t // PAGE >= held:  # the token opens or continues a new page
                if t % PAGE == 0:
                    wanted += 1
                    if wanted <= len(free):
                        tables[b, t // PAGE] = free[wanted - 1]
                        taken = wanted
                have = wanted <= len(free)
            else:
                have = True
            pos[row + k], own[row + k] = t, b
            if have:
                seq[b] = t + 1
                if tables[b, t // PAGE] >= 0:
                    slot[row + k] = tables[b, t // PAGE] * PAGE + t % PAGE
                else:
                    bad = True
            else:
                bad = True
        row += a
    cu[n] = row
    return dict(tables=tables, seq_lens=seq, cu_new=cu, positions=pos, slots=slot, row_seq=own, pages_used=taken, bad=bad)


# ---------------------------------------------------------------------------- rows
def rope_table(max_pos, theta=10000.0):
    a = np.arange(max_pos)[:, None] * theta ** (-np.arange(32) / 32)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def rotate(x, table_rows, interleaved):
    """x [..., 64] float64 turned by the rows [..., 64] of the fp32 table."""
    cs = table_rows.astype(np.float64)
    c, s = cs[..., :32], cs[..., 32:]
    i = np.arange(32)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
    out = np.empty_like(x)
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ia] * s + x[..., ib] * c
    return out


def rms(x, w, eps):
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def head_norm(x, w, b, eps):
    if w is None:
        return x
    if b is None:
        return rms(x, w, eps)
    x = x - x.mean(-1, keepdims=True)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w + b


def amax_scale(y):
    top = np.abs(y).max(-1)
    return np.where(top > 0, top / 448, 1.0)


# A value is computed in fp32 by a norm (a sum of n squares: at most n + 6
# roundings of a positive sum, half of that on the root) and a rotation (three
# roundings of terms that may cancel, and the table's own): under 2^-16 of the
# row's largest magnitude for rows of 512. Then it is rounded once.
FP32 = 2.0 ** -16


def check_bf16(got, ref):
    top = np.abs(ref).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + FP32 * top).all()


def check_e4m3(codes, scale, ref):
    """codes * scale against ref: half a step of e4m3 (2^-4 relative, 2^-10 of the scale below its normals)."""
    np.testing.assert_allclose(scale, amax_scale(ref), rtol=FP32)
    s = scale[..., None]
    assert (np.abs(codes * s - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) + 448 * FP32 * s).all()


# ---------------------------------------------------------------------------- attention
def attention_case(n_seqs, q, heads, kv_dtype, shared, seq_lens, seed=0, std=1.0, q_std=1.0, max_pages=None):
    """(cache, tables, seq_lens, q): shuffled pages; the page that holds the shared
    part's border is each request's own, and only row 0's holds the shared
    tokens (every other copy holds NaN there, as do all unused slots)."""
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-max(0, s) // PAGE)) for s in seq_lens]
    width = max(max(need), -(-shared // PAGE), 1) if max_pages is None else max_pages
    whole = shared // PAGE
    total = whole + sum(max(0, k - whole) for k in need) + -(-shared // PAGE) + 1
    perm = torch.randperm(total, generator=g).to(torch.int32)
    tables = torch.full((n_seqs, width), -1, dtype=torch.int32)
    at = whole
    for b in range(n_seqs):
        tables[b, :whole] = perm[:whole]
        last = max(need[b], -(-shared // PAGE) if b == 0 else 0)
        for p in range(whole, last):
            tables[b, p] = perm[at]
            at += 1
    cache = filled_cache(total, kv_dtype, seed + 1, std)
    live = torch.zeros(total, PAGE, dtype=torch.bool)
    for b in range(n_seqs):
        first, last = (0, max(seq_lens[b], shared)) if b == 0 else (shared, seq_lens[b])
        for s in range(first, last):
            live[tables[b, s // PAGE], s % PAGE] = True
    if kv_dtype == "bf16":
        cache.kv[~live] = float("nan")
    elif kv_dtype == "fp8":
        cache.kv[~live] = 0x7F
        cache.kv_scale[~live] = float("inf")
    else:
        cache.kv[~live] = 0xFF
    qt = (torch.randn(n_seqs * q, heads, D_QK, generator=g) * q_std).to(torch.bfloat16)
    return cache, tables, torch.tensor(seq_lens, dtype=torch.int32), qt


def attention_reference(cache, tables, seq_lens, q_per_seq, q, shared, sm_scale, bad_pages=()):
    """(out, lse, weight of |v|, largest sum |q||k| scale) in float64, a token at a time."""
    kv = latent_values(cache)
    rows, heads, _ = q.shape
    out = np.zeros((rows, heads, D_V))
    lse = np.full((rows, heads), -np.inf)
    mag = np.zeros((rows, heads, D_V))
    top = np.zeros((rows, heads))
    qd = q.float().double().numpy()
    for r in range(rows):
        b = r // q_per_seq
        n = max(0, int(seq_lens[b]) - q_per_seq + r % q_per_seq + 1)
        s = np.arange(n)
        page = tables.numpy()[np.where(s < shared, 0, b), s // PAGE]
        ok = (page >= 0) & (page < cache.kv.shape[0])
        k = kv[page[ok] * PAGE + s[ok] % PAGE]
        if not len(k):
            continue
        z = qd[r] @ k.T * sm_scale
        m = z.max(-1, keepdims=True)
        e = np.exp(z - m)
        l = e.sum(-1, keepdims=True)
        out[r], lse[r] = e / l @ k[:, :D_V], (m + np.log(l))[:, 0]
        mag[r] = e / l @ np.abs(k[:, :D_V])
        top[r] = (np.abs(qd[r]) @ np.abs(k).T * sm_scale).max(-1)
    return out, lse, mag, top


def check_attention(out, lse, ref, kv_dtype):
    """Every value within what its roundings can do.

    delta, the error of a logit: fp32 sums of 576 products (576 * 2^-24 of the
    sum of magnitudes), and for the tile-scaled rows their rounding to f16 (2^-11).
    Probabilities: rounded to bf16 (2^-8; f16 2^-11 for the tile-scaled rows,
    whose values are rounded as well), off by 2 delta from the logits (the
    maximum's too), fp32 sums over the keys (2^-14). The output is rounded to bf16."""
    ro, rl, mag, top = ref
    f16 = kv_dtype == "fp8_ds_mla"
    delta = top * (576 * 2.0 ** -24 + (2.0 ** -11 if f16 else 0.0)) + 2.0 ** -18
    rel = (2.0 ** -10 if f16 else 2.0 ** -8) + 2.0 ** -14 + 2 * delta
    out, lse = out.float().double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    err = np.abs(out - ro)
    bound = rel[..., None] * mag + 2.0 ** -8 * (np.abs(ro) + rel[..., None] * mag)
    worst = np.unravel_index(int(np.argmax(err - bound)), err.shape)
    assert (err <= bound).all(), f"value {worst}: {out[worst]} against {ro[worst]}"
    lerr = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl))
    lbound = delta + 2.0 ** -20 * np.abs(np.where(empty, 0, rl))
    assert (lerr <= lbound).all(), f"lse off by {lerr.max()}"


SM_SCALE = 1 / math.sqrt(D_QK)
