"""The serving entry points without a GPU: exported symbols, the binding's
checks, and the refusals of include/smla_serve.h, all before anything is
enqueued (the fake device pointers are never dereferenced). The references of
the GPU tests are checked against worked examples here."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import serve_common as sc

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "smla_serve.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    smla.build()
    return smla.lib()


def _cache(**kw):
    c = dict(kv=FAKE, kv_scale=FAKE, k_idx=FAKE, k_idx_scale=FAKE, num_pages=300, page_size=64,
             kv_dtype=smla.SMLA_FP8_E4M3, idx_dtype=smla.SMLA_FP8_E4M3, d_idx=128)
    c.update(kw)
    return smla.PagedCache(**c)


def test_header_symbols_exported(L):
    names = set(re.findall(r"^\s*(?:const\s+)?[\w]+\s*\**\s*(smla_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(smla._SERVE_SIGS)
    for n in names:
        assert hasattr(L, n)


def _tables(L, **kw):
    a = dict(ctx=FAKE, new=FAKE, n=4, tab=FAKE, mp=10, free=FAKE, nf=5, mx=100, seq=2 * FAKE, cu=FAKE, pos=FAKE, slots=FAKE,
             own=FAKE, used=FAKE, ws=FAKE, wsb=256)
    a.update(kw)
    return L.smla_build_tables(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(tab=None), INVALID), (dict(seq=None), INVALID),
    (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(used=None), INVALID), (dict(n=0), INVALID),
    (dict(mp=0), INVALID), (dict(mp=(1 << 25) + 1), UNSUPPORTED), (dict(nf=-1), INVALID), (dict(free=None), INVALID),
    (dict(mx=0), INVALID), (dict(seq=FAKE), INVALID), (dict(slots=FAKE + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=255), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE)])
def test_tables_refusals(L, kw, code):
    assert _tables(L, **kw) == code


def _append(L, cache=None, rope=None, **kw):
    a = dict(rows=7, slots=FAKE, pos=FAKE, ckv=FAKE, cs=576, kn=FAKE, k=FAKE, ks=128, w=FAKE, b=FAKE, eps=1e-6, ws=FAKE, wsb=256)
    a.update(kw)
    r = smla.RopeTable(FAKE, 100, 1, 0) if rope is None else rope
    return L.smla_cache_append(ctypes.byref(cache or _cache()), ctypes.byref(r), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(ckv=None, k=None), INVALID), (dict(rows=0), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID),
    (dict(ckv=FAKE + 8), INVALID), (dict(cs=570), INVALID), (dict(cs=580), INVALID), (dict(ks=120), INVALID),
    (dict(ks=129), INVALID), (dict(w=None), INVALID), (dict(kn=FAKE + 4), INVALID), (dict(b=FAKE + 8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(cache=_cache(page_size=32)), UNSUPPORTED),
    (dict(cache=_cache(kv=None)), INVALID), (dict(cache=_cache(kv_scale=None)), INVALID),
    (dict(cache=_cache(k_idx=None)), INVALID), (dict(cache=_cache(d_idx=64)), UNSUPPORTED),
    (dict(rope=smla.RopeTable(None, 100, 1, 0)), INVALID), (dict(rope=smla.RopeTable(FAKE, 0, 1, 0)), INVALID),
    (dict(rope=smla.RopeTable(FAKE + 4, 100, 1, 0)), INVALID)])
def test_append_refusals(L, kw, code):
    assert _append(L, **kw) == code


def _query(L, **kw):
    a = dict(rows=7, pos=FAKE, pe=FAKE, rs=64 * 192, hs=192, h=64, q=FAKE, raw=FAKE, raws=32 * 128, hi=32, di=128,
             dt=smla.SMLA_FP8_E4M3, nw=FAKE, eps=1e-6, w=FAKE, ws=1.0, qi=FAKE, wo=FAKE, wk=FAKE, wkb=256)
    a.update(kw)
    return L.smla_query_prep(ctypes.byref(smla.RopeTable(FAKE, 100, 1, 0)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(pe=None, raw=None), INVALID), (dict(rows=0), INVALID), (dict(pos=None), INVALID), (dict(q=None), INVALID),
    (dict(pe=FAKE + 2), INVALID), (dict(rs=12), INVALID), (dict(hs=60), INVALID), (dict(h=32), UNSUPPORTED),
    (dict(hi=12, raws=12 * 128), UNSUPPORTED), (dict(di=64), UNSUPPORTED), (dict(dt=smla.SMLA_BF16), UNSUPPORTED),
    (dict(dt=smla.SMLA_FP8_DS_MLA), INVALID), (dict(raws=4000), INVALID), (dict(w=None), INVALID), (dict(wo=None), INVALID),
    (dict(qi=None), INVALID), (dict(wk=None), WORKSPACE), (dict(wkb=128), WORKSPACE)])
def test_query_refusals(L, kw, code):
    assert _query(L, **kw) == code


def _attention(L, cache=None, **kw):
    a = dict(pt=FAKE, mp=40, n=3, lens=FAKE, mx=2500, sh=1000, q=2, qp=FAKE, h=64, sm=0.04, out=FAKE, lse=FAKE, ws=FAKE, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = L.smla_shared_prefix_fwd_workspace_size(a["n"], a["mx"], a["sh"], a["q"], a["h"], 1)
    return L.smla_shared_prefix_fwd(ctypes.byref(cache or _cache()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(pt=None), INVALID), (dict(lens=None), INVALID), (dict(qp=None), INVALID), (dict(out=None), INVALID),
    (dict(qp=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(n=0), INVALID),
    (dict(q=0), INVALID), (dict(mx=0), INVALID), (dict(mp=0), INVALID), (dict(mp=39), INVALID), (dict(sh=-1), INVALID),
    (dict(sh=2501), INVALID), (dict(sm=float("nan")), INVALID), (dict(h=32), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(wsb=255), WORKSPACE), (dict(cache=_cache(kv=None)), INVALID), (dict(cache=_cache(kv_scale=None)), INVALID),
    (dict(cache=_cache(kv_dtype=9)), INVALID), (dict(cache=_cache(page_size=16)), UNSUPPORTED)])
def test_attention_refusals(L, kw, code):
    assert _attention(L, **kw) == code


def test_attention_workspace_holds_the_wide_copy(L):
    size = lambda *a: L.smla_shared_prefix_fwd_workspace_size(*a)  # noqa: E731
    # 3 x 2 tokens x 64 heads = 3 row blocks share 1,000 tokens (16 pages of 64 rows of 1,152 bytes,
    # and four status words a page)
    for fp8 in (smla.SMLA_FP8_E4M3, smla.SMLA_FP8_DS_MLA):
        assert size(3, 2500, 1000, 2, 64, fp8) == size(3, 2500, 1000, 2, 64, smla.SMLA_BF16) + 16 * (64 * 1152 + 16)
        # one row block, or one request (nothing is shared), has none
        assert size(2, 2500, 1000, 1, 64, fp8) == size(2, 2500, 1000, 1, 64, smla.SMLA_BF16)
        assert size(1, 2500, 1000, 9, 64, fp8) == size(1, 2500, 1000, 9, 64, smla.SMLA_BF16)
    need = size(3, 2500, 1000, 2, 64, smla.SMLA_FP8_E4M3)
    assert _attention(L, wsb=need - 1) == WORKSPACE


def test_binding_refuses_wrong_tensors(L):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        smla.build_tables(i(3).long(), i(3), i(3, 4), i(2), 8, ws=torch.zeros(256, dtype=torch.uint8), stream=0)
    with pytest.raises(ValueError):
        smla.build_tables(i(2), i(3), i(3, 4), i(2), 8, ws=torch.zeros(256, dtype=torch.uint8), stream=0)
    c = sc.empty_cache(2)
    rope = sc.rope_table(10)
    with pytest.raises(ValueError):
        smla.cache_append(c, i(4), i(3), rope, ckv=torch.zeros(4, 576, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        smla.cache_append(c, i(4), i(4), rope, ckv=torch.zeros(4, 576), stream=0)
    with pytest.raises(ValueError):
        smla.cache_append(c, i(4), i(4), rope.double(), ckv=torch.zeros(4, 576, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        smla.query_prep(i(4), rope, q_pe=torch.zeros(4, 64, 192, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        smla.shared_prefix_fwd(c, i(2, 4), i(2), 100, 50, 1, torch.zeros(3, 64, 576, dtype=torch.bfloat16), 0.04, stream=0)


def test_tables_reference_worked_example():
    # two requests: 62 tokens + 4 (two in the held page 9, two in a new one), 64 + 1 (a new page), then an idle one
    r = sc.tables_reference(np.array([62, 64, 5]), np.array([4, 1, 0]), np.array([[9, -1], [3, -1], [7, -1]], np.int32),
                            np.array([20, 21, 22]), 7)
    assert r["tables"].tolist() == [[9, 20], [3, 21], [7, -1]]
    assert r["slots"].tolist() == [9 * 64 + 62, 9 * 64 + 63, 20 * 64, 20 * 64 + 1, 21 * 64, -1, -1]
    assert r["positions"].tolist() == [62, 63, 64, 65, 64, -1, -1]
    assert r["seq_lens"].tolist() == [66, 65, 5] and r["cu_new"].tolist() == [0, 4, 5, 5] and r["pages_used"] == 2
    assert not r["bad"]


def test_rotation_reference_turns_by_the_angle():
    t = sc.rope_table(9).numpy()
    x = np.zeros(64)
    x[0] = 1.0  # the first of pair 0 under both pairings: angle = position
    for inter, other in ((True, 1), (False, 32)):
        y = sc.rotate(x, t[5], inter)
        assert abs(y[0] - np.cos(5)) < 1e-6 and abs(y[other] - np.sin(5)) < 1e-6 and np.count_nonzero(y) == 2


def test_attention_reference_equals_softmax():
    c, tab, lens, q = sc.attention_case(2, 2, 16, "bf16", 70, [75, 91], seed=3)
    out, lse, _, _ = sc.attention_reference(c, tab, lens, 2, q, 70, sc.SM_SCALE)
    kv = c.kv.double().view(-1, 576)
    s = torch.arange(91)
    k = kv[tab[torch.where(s < 70, 0, 1), s // 64].long() * 64 + s % 64]
    z = q[3].double() @ k.T * sc.SM_SCALE
    assert np.allclose(out[3], (z.softmax(-1) @ k[:, :512]).numpy(), atol=1e-12)
    assert np.allclose(lse[3], z.logsumexp(-1).numpy(), atol=1e-12)
