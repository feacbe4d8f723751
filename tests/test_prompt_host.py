"""The expanded-prompt entry points without a GPU: exported symbols, the refusals of include/smla_prompt.h
(before anything is enqueued: the fake device pointers are never dereferenced), the binding's checks, and the
references of the GPU tests against worked examples."""
import ctypes
import math
import os
import re

import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import prompt_common as pc

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "smla_prompt.h")
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE, NAN, INF = 0x10000, float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    smla.build()
    return smla.lib()


def test_header_symbols_exported(L):
    names = set(re.findall(r"^\s*(?:const\s+)?[\w]+\s*\**\s*(smla_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(smla._PROMPT_SIGS)
    for n in names:
        assert hasattr(L, n)


def _table(L, **kw):
    a = dict(out=FAKE, first=0, n=10, dim=64, base=1e4, factor=1.0, orig=0, fast=32.0, slow=1.0, mag=1.0)
    a.update(kw)
    return L.smla_rope_table(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(n=0), INVALID), (dict(first=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dim=12), UNSUPPORTED), (dict(dim=264), UNSUPPORTED), (dict(base=1.0), INVALID), (dict(base=NAN), INVALID), (dict(base=INF), INVALID),
    (dict(factor=0.5), INVALID), (dict(factor=NAN), INVALID), (dict(factor=INF), INVALID), (dict(mag=NAN), INVALID), (dict(orig=-1), INVALID),
    (dict(orig=4096, slow=0.0), INVALID), (dict(orig=4096, fast=0.5), INVALID), (dict(orig=4096, fast=NAN), INVALID),
    (dict(first=(1 << 31) - 9), UNSUPPORTED)])
def test_table_refusals(L, kw, code):
    assert _table(L, **kw) == code


def _rope(L, **kw):
    a = dict(cs=FAKE, mp=100, dim=64, inter=1, rows=5, pos=FAKE, x=FAKE, xr=64 * 192, xh=192, h=64, out=2 * FAKE, outr=64 * 64, outh=64,
             ws=FAKE, wsb=256)
    a.update(kw)
    return L.smla_rope_apply(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(cs=None), INVALID), (dict(pos=None), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(cs=FAKE + 8), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID), (dict(pos=FAKE + 2), INVALID), (dict(mp=0), INVALID), (dict(rows=0), INVALID),
    (dict(h=0), INVALID), (dict(dim=0), INVALID), (dict(dim=20), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(xr=12), INVALID),
    (dict(xh=60), INVALID), (dict(xh=56), INVALID), (dict(outh=32), INVALID), (dict(xr=-64), INVALID), (dict(outr=32), INVALID),
    (dict(out=FAKE), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=128), WORKSPACE), (dict(ws=FAKE + 4), WORKSPACE)])
def test_rope_refusals(L, kw, code):
    assert _rope(L, **kw) == code


def _cache(**kw):
    c = dict(kv=FAKE, kv_scale=FAKE, k_idx=FAKE, k_idx_scale=FAKE, num_pages=300, page_size=64,
             kv_dtype=smla.SMLA_FP8_E4M3, idx_dtype=smla.SMLA_FP8_E4M3, d_idx=128)
    c.update(kw)
    return smla.PagedCache(**c)


def _read(L, cache=None, **kw):
    a = dict(pt=FAKE, mp=40, n=3, cu=FAKE, rows=100, st=FAKE, lat=FAKE, ls=512, pe=FAKE, ps=64, keys=FAKE, ks=128, ws=FAKE, wsb=256)
    a.update(kw)
    return L.smla_cache_read(ctypes.byref(cache or _cache()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(lat=None, pe=None, keys=None), INVALID), (dict(pt=None), INVALID), (dict(cu=None), INVALID), (dict(mp=0), INVALID),
    (dict(n=0), INVALID), (dict(rows=0), INVALID), (dict(rows=(1 << 31) - 1), UNSUPPORTED), (dict(n=(1 << 31) - 1), UNSUPPORTED),
    (dict(ls=504), INVALID), (dict(ls=516), INVALID), (dict(lat=FAKE + 8), INVALID), (dict(ps=56), INVALID), (dict(pe=FAKE + 2), INVALID),
    (dict(ks=120), INVALID), (dict(st=FAKE + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(cache=_cache(kv=None)), INVALID), (dict(cache=_cache(kv_scale=None)), INVALID), (dict(cache=_cache(k_idx=None)), INVALID),
    (dict(cache=_cache(page_size=32)), UNSUPPORTED), (dict(cache=_cache(kv_dtype=7)), INVALID), (dict(cache=_cache(d_idx=64)), UNSUPPORTED)])
def test_read_refusals(L, kw, code):
    assert _read(L, **kw) == code


def _prompt(L, **kw):
    a = dict(q=smla.Heads(FAKE, 64 * 192, 192), k=smla.Heads(FAKE, 64 * 256, 256), v=smla.Heads(FAKE, 64 * 256, 256), pe=FAKE, ps=64, tq=100,
             tk=300, n=3, cq=FAKE, ck=FAKE, h=64, hk=64, d=192, causal=1, sm=0.07, po=None, pl=None, out=FAKE, f32=0, lse=FAKE, ws=FAKE, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = L.smla_prompt_fwd_workspace_size(a["tq"], a["tk"], a["n"], a["h"], a["hk"])
    heads = [None if a[x] is None else ctypes.byref(a[x]) for x in ("q", "k", "v")]
    return L.smla_prompt_fwd(*heads, *list(a.values())[3:], None)


def _h(*a):
    return smla.Heads(*a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=_h(None, 64 * 192, 192)), INVALID),
    (dict(q=_h(FAKE + 8, 64 * 192, 192)), INVALID), (dict(q=_h(FAKE, 64 * 192, 184)), INVALID), (dict(q=_h(FAKE, 64 * 192, 196)), INVALID),
    (dict(q=_h(FAKE, 184, 192)), INVALID), (dict(k=_h(FAKE, 64 * 256 + 4, 256)), INVALID), (dict(k=_h(FAKE, 64 * 256, 120)), INVALID),
    (dict(v=_h(FAKE, 64 * 256, 0)), INVALID), (dict(v=_h(FAKE, 1 << 35, 256)), INVALID), (dict(v=_h(FAKE, 64 * 256, 1 << 35)), INVALID),
    (dict(pe=FAKE + 2), INVALID), (dict(ps=56), INVALID), (dict(ps=68), INVALID), (dict(tq=0), INVALID), (dict(tk=0), INVALID), (dict(n=0), INVALID),
    (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(cq=FAKE + 2), INVALID), (dict(h=0), INVALID), (dict(hk=0), INVALID),
    (dict(hk=48), INVALID), (dict(h=2048, hk=64), UNSUPPORTED), (dict(d=64), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(sm=NAN), INVALID), (dict(sm=INF), INVALID), (dict(po=2 * FAKE), INVALID), (dict(pl=2 * FAKE), INVALID),
    (dict(po=2 * FAKE + 8, pl=2 * FAKE), INVALID), (dict(po=FAKE, pl=2 * FAKE), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(tq=(1 << 31) - 1), UNSUPPORTED), (dict(tk=(1 << 31) - 1), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=FAKE + 8), WORKSPACE), (dict(wsb=255), WORKSPACE)])
def test_prompt_refusals(L, kw, code):
    assert _prompt(L, **kw) == code


def test_prompt_workspace_is_needed_in_full(L):
    need = L.smla_prompt_fwd_workspace_size(100, 30000, 3, 64, 64)
    assert need >= 256 and _prompt(L, tk=30000, wsb=need - 1) == WORKSPACE


def test_binding_refuses_wrong_tensors(L):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):  # not on the GPU
        smla.rope_table(4, out=torch.zeros(4, 64), stream=0)
    with pytest.raises(ValueError):
        smla.rope_table(4, out=torch.zeros(4, 32), stream=0)
    for x, pos, tab in ((b(4, 2, 64), i(3), torch.zeros(9, 64)), (b(4, 2, 64).float(), i(4), torch.zeros(9, 64)),
                        (b(4, 2, 64), i(4).long(), torch.zeros(9, 64)), (b(4, 2, 64), i(4), torch.zeros(9, 32)),
                        (b(4, 64, 2).mT, i(4), torch.zeros(9, 64)), (b(4, 2, 64), i(4), torch.zeros(9, 64))):
        with pytest.raises(ValueError):
            smla.rope_apply(x, pos, tab, stream=0)
    for c, kw in ((i(3), {}), (i(4), dict(starts=i(2))), (i(4), dict(latent=b(8, 500))), (i(4).long(), {}), (i(4), {})):
        with pytest.raises(ValueError):
            smla.cache_read(_TinyCache(), i(3, 4), c, 8, stream=0, **kw)
    q, k, v = b(4, 2, 192), b(6, 2, 128), b(6, 2, 128)
    for args, kw in (((q, k, v, i(3), i(3)), {}), ((q, k, v, i(3), i(2)), dict(k_pe=b(6, 64))), ((q, k, b(5, 2, 128), i(3), i(3)), dict(k_pe=b(6, 64))),
                     ((q.float(), k, v, i(3), i(3)), dict(k_pe=b(6, 64))), ((q, k, v, i(3), i(3)), dict(k_pe=b(6, 32))),
                     ((q, k, v, i(3), i(3)), dict(k_pe=b(6, 64), out=b(4, 2, 64))), ((q, k, v, i(3), i(3)), dict(k_pe=b(6, 64), prev_out=b(4, 2, 128))),
                     ((q, k, v, i(3), i(3)), dict(k_pe=b(6, 64)))):
        with pytest.raises(ValueError):
            smla.prompt_fwd(*args, 0.1, stream=0, **kw)


class _TinyCache:
    kv, kv_scale = torch.zeros(2, 64, 576, dtype=torch.uint8), torch.zeros(2, 64)
    k_idx, k_idx_scale, kv_dtype, idx_dtype = torch.zeros(2, 64, 128, dtype=torch.uint8), torch.zeros(2, 64), "fp8", "fp8"


def test_frequency_reference():
    w = pc.frequencies(64, factor=8.0, original=4096)
    plain = pc.frequencies(64)
    assert w[0] == plain[0] and abs(w[-1] / (plain[-1] / 8) - 1) < 1e-12  # fast pairs as they are, slow ones by the factor
    assert ((w <= plain) & (w >= plain / 8)).all()
    assert torch.equal(pc.frequencies(64, factor=4.0), plain / 4)


def test_attention_reference():
    q, k, v, pe, cq, ck = pc.prompt_case([2, 3], [4, 3], 4, 2, 192, True, seed=1)
    out, lse, _, _, _ = pc.prompt_reference(q, k, v, pe, cq, ck, 0.1, True)
    # the first request's second token, head 3, sees keys 0..3 of key head 1
    z = (q[1, 3, :128].double() @ k[:4, 1].double().T + q[1, 3, 128:].double() @ pe[:4].double().T) * 0.1
    assert torch.allclose(out[1, 3], torch.softmax(z, 0) @ v[:4, 1].double()) and abs(lse[1, 3] - torch.logsumexp(z, 0)) < 1e-12
    assert torch.allclose(out[2, 0], v[4, 0].double())  # the second request's first token sees one key
    # two halves of the keys, joined, are the whole
    args = (q[:2], k[:2], v[:2], pe[:2], pc.cu([2]), pc.cu([2]), 0.1, False)
    a = pc.prompt_reference(*args)
    whole = pc.prompt_reference(q[:2], k[:4], v[:4], pe[:4], pc.cu([2]), pc.cu([4]), 0.1, False)
    both = pc.prompt_reference(q[:2], k[2:4], v[2:4], pe[2:4], pc.cu([2]), pc.cu([2]), 0.1, False, prev=a[:2])
    assert torch.allclose(both[0], whole[0]) and torch.allclose(both[1], whole[1])
    none = pc.prompt_reference(q[:5], k, v, pe, pc.cu([5]), pc.cu([3]), 0.1, True)
    assert (none[0][:2] == 0).all() and none[1][:2].isneginf().all() and math.isfinite(none[1][2, 0])
