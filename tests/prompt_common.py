"""Inputs, 64-bit references and derived bounds of the expanded-prompt operators' tests (plain torch in
float64, written from the formulas; nothing of the package's kernels)."""
import math

import torch

BF16 = 2.0 ** -8   # half a step, relative
FP32 = 2.0 ** -24


def cu(lens, device="cpu"):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).to(device)


# ---------------------------------------------------------------------------- rotation
def frequencies(dim, base=10000.0, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, one at a time."""
    out = []
    for i in range(dim // 2):
        w = base ** (-2.0 * i / dim)
        if original == 0:
            out.append(w / factor)
            continue
        edge = lambda beta: dim * math.log(original / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(edge(beta_fast)), 0), min(math.ceil(edge(beta_slow)), dim - 1)
        r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(w * (1 - r) + w / factor * r)
    return torch.tensor(out, dtype=torch.float64)


def table_reference(n, dim, first=0, magnitude=1.0, **kw):
    a = torch.arange(first, first + n, dtype=torch.float64)[:, None] * frequencies(dim, **kw)
    return magnitude * torch.cat([a.cos(), a.sin()], 1)


def rotate(x, rows, interleaved):
    """x [.., dim] float64 turned by the table rows [.., dim]; (result, |a| + |b| of each value's pair)."""
    h = x.shape[-1] // 2
    i = torch.arange(h)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    c, s = rows[..., :h].double(), rows[..., h:].double()
    out, mag = torch.empty_like(x), torch.empty_like(x)
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ia] * s + x[..., ib] * c
    mag[..., ia] = mag[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return out, mag


def check_rotated(got, ref, mag):
    """Two products and a sum in fp32 (three roundings of at most |a| + |b| times a table value of up to 1), rounded once to bf16."""
    assert ((got.double() - ref).abs() <= BF16 * ref.abs() + 4 * FP32 * mag).all()


# ---------------------------------------------------------------------------- attention
def prompt_case(ql, kl, heads, kv_heads, d, pe, seed=0, extra_q=0, extra_k=0, std=1.0):
    """(q, k, v, k_pe, cu_q, cu_k): a head's keys and values side by side as an up-projection leaves them;
    extra rows behind the last request hold NaN."""
    g = torch.Generator().manual_seed(seed)
    tq, tk = max(1, sum(ql) + extra_q), max(1, sum(kl) + extra_k)
    dk = d - 64 if pe else d
    kv = torch.randn(tk, kv_heads, dk + 128, generator=g).to(torch.bfloat16)
    q = (torch.randn(tq, heads, d, generator=g) * std).to(torch.bfloat16)
    p = torch.randn(tk, 64, generator=g).to(torch.bfloat16) if pe else None
    q[sum(ql):], kv[sum(kl):] = float("nan"), float("nan")
    if pe:
        p[sum(kl):] = float("nan")
    return q, kv[..., :dk], kv[..., dk:], p, cu(ql), cu(kl)


def prompt_reference(q, k, v, pe, cq, ck, scale, causal, prev=None):
    """(out, lse, sum of p |v|, largest sum |q||k| scale, most keys), a request and a head at a time, on q's device."""
    f, dev = torch.float64, q.device
    heads, kv_heads = q.shape[1], k.shape[1]
    out = torch.zeros(q.shape[0], heads, 128, dtype=f, device=dev)
    mag, lse = torch.zeros_like(out), torch.full((q.shape[0], heads), -math.inf, dtype=f, device=dev)
    top = torch.zeros_like(lse)
    cq, ck = cq.tolist(), ck.tolist()
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if nq <= 0 or nk <= 0:
            continue
        rows, keys = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        pos = torch.arange(nq, device=dev)[:, None] + nk - nq
        hidden = torch.arange(nk, device=dev)[None] > pos if causal else torch.zeros(nq, nk, dtype=torch.bool, device=dev)
        any_key = ~hidden.all(1)
        for h in range(heads):
            g = h // (heads // kv_heads)
            kh = k[keys, g].to(f)
            if pe is not None:
                kh = torch.cat([kh, pe[keys].to(f)], 1)
            qh, vh = q[rows, h].to(f), v[keys, g].to(f)
            z = (qh @ kh.T * scale).masked_fill(hidden, -math.inf)
            w = torch.softmax(z, 1).masked_fill(hidden, 0.0)
            # a hidden key's value may be anything: it is not multiplied by its zero
            o = w @ torch.nan_to_num(vh, 0.0, 0.0, 0.0)
            for j in (~torch.isfinite(vh)).any(1).nonzero().flatten().tolist():
                sees = ~hidden[:, j]
                bad = ~torch.isfinite(vh[j])
                o[sees[:, None] & bad[None]] += (sees[:, None] * vh[j][None])[sees[:, None] & bad[None]]
            out[rows, h] = torch.where(any_key[:, None], o, 0.0)
            lse[rows, h] = torch.where(any_key, torch.logsumexp(z, 1), -math.inf)
            mag[rows, h] = torch.where(any_key[:, None], w @ torch.nan_to_num(vh, 0.0, 0.0, 0.0).abs(), 0.0)
            top[rows, h] = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(1)
    if prev is not None:
        po, pl = prev[0].to(f), prev[1].to(f)
        both = torch.logaddexp(pl, lse)
        wp, wo = (pl - both).exp().nan_to_num(0.0), (lse - both).exp().nan_to_num(0.0)
        po = torch.where(torch.isneginf(pl)[..., None], 0.0, po)
        out = wp[..., None] * po + wo[..., None] * out
        mag = wp[..., None] * po.abs() + wo[..., None] * mag
        lse = both
    return out, lse, mag, top, max([0] + [b - a for a, b in zip(ck, ck[1:])])


def check_prompt(out, lse, ref, rows=None):
    """Every value within what its roundings can do.

    delta, the error of a logit: a sum of up to 192 products in fp32 (2 * 192 * 2^-24 of the sum of the
    magnitudes, were every sum cut instead of rounded) and the exponent's and the scale's own (2^-18).
    Probabilities: rounded to bf16 (2^-8), off by 2 delta from the logits (the maximum's too); their sums
    and their product with V run over the keys in fp32 (2^-23 a key, cut instead of rounded, against the sum of
    the magnitudes). Joining with other results: some roundings more of fp32 (2^-18). Then bf16 rounds once."""
    ro, rl, mag, top, keys = (t if rows is None or not torch.is_tensor(t) else t[rows] for t in ref)
    out_t = out.dtype
    out, lse = out.double().to(ro.device), lse.double().to(ro.device)
    if rows is not None:
        out, lse = out[rows], lse[rows]
    delta = top * (2 * 192 * FP32) + 2.0 ** -18
    rel = (BF16 + 2 * FP32 * keys + 2 * delta + 2.0 ** -18)[..., None]
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    last = BF16 if out_t == torch.bfloat16 else FP32
    err, bound = (out - ro).abs(), rel * mag + last * (ro.abs() + rel * mag)
    same = torch.isfinite(ro)
    assert (err[same] <= bound[same]).all(), f"off by up to {float((err - bound)[same].max())} more than its bound"
    odd = ~same
    assert torch.equal(out[odd].isnan(), ro[odd].isnan()) and torch.equal(out[odd].isposinf(), ro[odd].isposinf())
    lerr, real = (lse - rl).abs(), ~empty & torch.isfinite(rl)
    assert (lerr[real] <= (delta + 2 * FP32 * keys + 2.0 ** -20 * rl.abs())[real]).all(), f"lse off by {float(lerr[real].max())}"
