"""Prefills of one to eight tokens (the rest of a chunked prompt, for instance), which decode-shaped calls take in another
mode of the indexer: against the CPU oracle, index sets exactly."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import oracle
from indexer_top_sparse_score_gb300 import workloads as wl
from tests.gpu_common import compare_idx, compare_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    smla.build()
    oracle.build()


def _spec(h_idx, n, prefix, **kw):
    if h_idx == 4:
        return wl.scaled(wl.SPECS["tiny"], n_tokens=n, prefix_len=prefix, shuffled=True, **kw)
    return wl.scaled(wl.SPECS["prefill16k"], n_tokens=n, prefix_len=prefix, shuffled=True, h_idx=h_idx, topk=512, **kw)


def _check(prob, out, lse, idx=None):
    ridx, _, rout, rlse, _, bad = oracle.Oracle(prob).rows(np.arange(prob.spec.n_tokens))
    assert not bad.any()
    if idx is not None:
        compare_idx(idx.cpu().numpy(), ridx)
    compare_out(out.float().cpu().numpy(), rout, lse.cpu().numpy(), rlse, prob.spec.kv_dtype)


@pytest.mark.parametrize("prefix", [0, 5, 700, 17000])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("h_idx", [4, 8, 16, 32, 64])
def test_short_prefill(h_idx, n, prefix):
    prob = wl.make(_spec(h_idx, n, prefix, **({"kv_dtype": "fp8"} if n % 2 else {})), "cpu")
    spec, dev = prob.spec, prob.to("cuda")
    for full in (True, False):  # the whole workspace, and the smallest one
        ws = None if full else smla.workspace(256 + n * spec.topk * 4)
        idx = torch.full((n, spec.topk), -7, dtype=torch.int32, device="cuda") if full else None
        out, lse, _, ws = smla.sparse_mla_prefill(dev.cache, dev.page_table, prefix, dev.q, dev.q_idx, dev.w, spec.topk, spec.sm_scale,
                                                  out_idx=idx, ws=ws)
        assert smla.read_status(ws)[0] == 0
        _check(prob, out, lse, idx)


@pytest.mark.parametrize("n,chunk", [(1025, 1024), (303, [300, 3])])
def test_host_prefill_with_a_short_last_chunk(n, chunk):
    prob = wl.make(_spec(32, n, 100), "cpu")
    spec, dev = prob.spec, prob.to("cuda")
    hp = smla.HostPrefill(dev.cache, dev.page_table, 100, n, spec.n_heads, spec.h_idx, spec.d_idx, spec.idx_dtype, spec.topk, spec.sm_scale,
                          chunk=chunk)
    out, lse = torch.empty((n, spec.n_heads, 512), dtype=torch.bfloat16).pin_memory(), torch.empty((n, spec.n_heads)).pin_memory()
    hp.run(prob.q.pin_memory(), prob.q_idx.pin_memory(), prob.w.pin_memory(), out, lse)
    assert hp.read_status() == (0, 0)
    rows = np.array([0, n // 2, n - 3, n - 2, n - 1])
    _, _, rout, rlse, _, bad = oracle.Oracle(prob).rows(rows)
    assert not bad.any()
    compare_out(out.float().numpy()[rows], rout, lse.numpy()[rows], rlse, spec.kv_dtype)


def test_short_prefill_without_a_workspace():
    import ctypes
    prob = wl.make(_spec(32, 3, 900), "cpu")
    spec, dev = prob.spec, prob.to("cuda")
    out, lse = torch.empty((3, spec.n_heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((3, spec.n_heads), device="cuda")
    L, c, bits = smla.lib(), smla.make_cache(dev.cache), ctypes.c_uint32(0)
    st = torch.cuda.current_stream().cuda_stream
    rc = L.smla_sparse_mla_prefill_noalloc(ctypes.byref(c), dev.page_table.data_ptr(), 900, 3, dev.q.data_ptr(), spec.n_heads, dev.q_idx.data_ptr(),
                                           dev.w.data_ptr(), spec.h_idx, spec.topk, spec.sm_scale, out.data_ptr(), lse.data_ptr(), st)
    assert rc == 0 and L.smla_noalloc_read_status(st, ctypes.byref(bits)) == 0 and bits.value == 0
    _check(prob, out, lse)
