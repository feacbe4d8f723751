"""The serving operators on the GPU against 64-bit references (serve_common)."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import serve_common as sc

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


# ---------------------------------------------------------------------------- tables
def _run_tables(ctx, new, tables, free, max_new):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    tab = d(tables)
    seq, cu, pos, slots, own, used, ws = smla.build_tables(d(ctx), d(new), tab, d(free), max_new)
    rc, _ = smla.read_status(ws)
    h = lambda t: t.cpu().numpy()  # noqa: E731
    return dict(tables=h(tab), seq_lens=h(seq), cu_new=h(cu), positions=h(pos), slots=h(slots), row_seq=h(own),
                pages_used=int(used), bad=rc != 0)


def _same(got, ref):
    for k, v in ref.items():
        assert np.array_equal(got[k], v), k


def _random_tables(n, ctx_max, new_max, seed, n_free=None, extra_cols=1):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_max + 1, n), rng.integers(0, new_max + 1, n)
    width = -(-(ctx_max + new_max) // 64) + extra_cols
    nf = n * (new_max // 64 + 2) if n_free is None else n_free
    ids = rng.permutation(n * width + nf)
    tables = np.where(np.arange(width)[None] < -(-ctx[:, None] // 64), ids[nf:].reshape(n, width), -1)
    return ctx, new, tables, ids[:nf]


@pytest.mark.parametrize("n,ctx_max,new_max", [(1, 0, 1), (1, 63, 1), (1, 64, 1), (3, 200, 130), (64, 131000, 2), (255, 300, 3),
                                               (256, 300, 3), (257, 300, 3), (1000, 5000, 70), (2, 100, 9000),
                                               (1023, 90, 5), (1024, 90, 5), (1025, 90, 5), (3001, 200, 40)])
def test_tables(n, ctx_max, new_max):
    ctx, new, tables, free = _random_tables(n, ctx_max, new_max, n + ctx_max)
    for max_new in (max(1, int(new.sum())), int(new.sum()) + 777):
        _same(_run_tables(ctx, new, tables, free, max_new), sc.tables_reference(ctx, new, tables, free, max_new))


def test_tables_all_idle():
    ctx, new, tables, free = _random_tables(70, 500, 0, 5)
    _same(_run_tables(ctx, new, tables, free, 16), sc.tables_reference(ctx, new, tables, free, 16))


@pytest.mark.parametrize("n_free", [0, 1, 7])
def test_tables_free_list_runs_out(n_free):
    ctx, new, tables, free = _random_tables(40, 300, 200, 11, n_free=n_free)
    ref = sc.tables_reference(ctx, new, tables, free, int(new.sum()))
    assert ref["bad"]
    _same(_run_tables(ctx, new, tables, free, int(new.sum())), ref)


def test_tables_reports_bad_lengths_and_overflow():
    ctx, new, tables, free = _random_tables(9, 300, 100, 12)
    ctx[2], new[4], new[6] = -5, -1, 10 ** 6
    ref = sc.tables_reference(ctx, new, tables, free, 250)
    assert ref["bad"] and ref["seq_lens"][2] == ref["seq_lens"][6] == 0
    _same(_run_tables(ctx, new, tables, free, 250), ref)


def test_tables_missing_held_page():
    ctx, new, tables, free = _random_tables(5, 300, 100, 13)
    ctx[1], new[1] = 70, 5
    tables[1, 1] = -1
    ref = sc.tables_reference(ctx, new, tables, free, int(new.sum()))
    assert ref["bad"]
    _same(_run_tables(ctx, new, tables, free, int(new.sum())), ref)


# ---------------------------------------------------------------------------- rows
def _rows(n, width, seed, std=1.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, width + pad, generator=g) * std).to(torch.bfloat16)[:, :width]


def _weights(n, seed, mean):
    g = torch.Generator().manual_seed(seed)
    return mean + 0.1 * torch.randn(n, generator=g)


def _slots(rows, pages, seed, holes):
    g = torch.Generator().manual_seed(seed)
    s = torch.randperm(pages * 64, generator=g)[:rows].to(torch.int32)
    if holes:
        s[::3] = -1
    return s


def _cu(t):
    return None if t is None else t.cuda()


def _strided_cuda(t):
    """On the GPU with the row stride that t has here."""
    if t is None:
        return None
    base = torch.empty(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")
    base[:, :t.shape[1]] = t.cuda()
    return base[:, :t.shape[1]]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("idx_dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows,inter,norm,holes,pad", [(1, True, True, False, 0), (3, False, True, True, 0), (130, True, False, True, 64),
                                                       (515, False, True, False, 8)])
def test_append(kv_dtype, idx_dtype, rows, inter, norm, holes, pad):
    pages = rows // 64 + 2
    d = 128 if idx_dtype == "fp8" else 64
    c = sc.empty_cache(pages, kv_dtype, idx_dtype, fill=0x5A).to("cuda")
    ckv, kr = _rows(rows, 576, rows, pad=pad), _rows(rows, d, rows + 1, pad=pad)
    ckv[0] = 0  # a row of zeros: scale 1
    kn, iw, ib = (_weights(512, 1, 1.0), _weights(d, 2, 1.0), _weights(d, 3, 0.0)) if norm else (None, None, None)
    slots, rope = _slots(rows, pages, 4, holes), sc.rope_table(1000)
    pos = torch.randint(0, 1000, (rows,), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    before = [None if t is None else t.clone() for t in (c.kv, c.kv_scale, c.k_idx, c.k_idx_scale)]
    ws = smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), ckv=_strided_cuda(ckv), kv_norm=_cu(kn), k_idx=_strided_cuda(kr),
                           idx_norm=_cu(iw), idx_bias=_cu(ib), eps=EPS, kv_interleaved=inter, idx_interleaved=not inter)
    assert smla.read_status(ws)[0] == 0
    n64 = lambda t: None if t is None else t.float().double().numpy()  # noqa: E731
    turns = rope.numpy()[pos.numpy()]
    x = n64(ckv)
    lat, pe = sc.rms(x[:, :512], n64(kn), EPS), sc.rotate(x[:, 512:], turns, inter)
    key = sc.head_norm(n64(kr), n64(iw), n64(ib), EPS)
    key[:, :64] = sc.rotate(key[:, :64], turns, not inter)
    live = (slots >= 0).numpy()
    at = slots.numpy()[live].astype(np.int64)
    kv = c.kv.cpu().reshape(pages * 64, -1)[at]
    f8 = lambda b: b.contiguous().view(torch.float8_e4m3fn).float().double().numpy()  # noqa: E731
    if kv_dtype == "bf16":
        sc.check_bf16(n64(kv)[:, :512], lat[live])
        sc.check_bf16(n64(kv)[:, 512:], pe[live])
    elif kv_dtype == "fp8":
        sc.check_e4m3(f8(kv), c.kv_scale.cpu().double().numpy().reshape(-1)[at], np.concatenate([lat, pe], 1)[live])
    else:
        s = kv[:, 512:528].contiguous().view(torch.float32).double().numpy()
        sc.check_e4m3(f8(kv[:, :512]).reshape(-1, 4, 128), s, lat[live].reshape(-1, 4, 128))
        sc.check_bf16(n64(kv[:, 528:].contiguous().view(torch.bfloat16)), pe[live])
    ki = c.k_idx.cpu().reshape(pages * 64, -1)[at]
    if idx_dtype == "bf16":
        sc.check_bf16(n64(ki), key[live])
    else:
        sc.check_e4m3(f8(ki), c.k_idx_scale.cpu().double().numpy().reshape(-1)[at], key[live])
    rest = np.setdiff1d(np.arange(pages * 64), at)  # nothing else is touched
    for t, b in zip((c.kv, c.kv_scale, c.k_idx, c.k_idx_scale), before):
        if t is not None:
            a, b = (v.reshape(pages * 64, -1).contiguous().view(torch.uint8).cpu().numpy()[rest] for v in (t, b))
            assert np.array_equal(a, b)


def test_append_parts_and_plain_keys():
    """Only one of the two kinds of rows; RMS norm without bias; e4m3 keys without a scale saturate."""
    rows, c = 70, sc.empty_cache(3, "bf16", "fp8", key_scale=False).to("cuda")
    kr, iw, rope = _rows(rows, 128, 7, std=200.0), _weights(128, 8, 1.0), sc.rope_table(70)
    slots, pos = _slots(rows, 3, 9, False), torch.arange(rows, dtype=torch.int32)
    smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), k_idx=_cu(kr), eps=EPS)
    assert not c.kv.any()
    key = kr.float().double().numpy()
    key[:, :64] = sc.rotate(key[:, :64], rope.numpy(), False)
    at = slots.numpy()
    got = c.k_idx.cpu().view(torch.float8_e4m3fn).float().double().numpy().reshape(-1, 128)[at]
    ref = np.clip(key, -448, 448)
    assert (np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10) + sc.FP32 * np.abs(key).max(-1, keepdims=True)).all()
    smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), k_idx=_cu(kr), idx_norm=_cu(iw), eps=EPS)
    key = sc.rms(kr.float().double().numpy(), iw.double().numpy(), EPS)
    key[:, :64] = sc.rotate(key[:, :64], rope.numpy(), False)
    got = c.k_idx.cpu().view(torch.float8_e4m3fn).float().double().numpy().reshape(-1, 128)[at]
    assert (np.abs(got - key) <= np.maximum(2.0 ** -4 * np.abs(key), 2.0 ** -10) + sc.FP32 * np.abs(key).max(-1, keepdims=True)).all()
    before = c.k_idx.clone()
    smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), ckv=_cu(_rows(rows, 576, 10)), eps=EPS)
    assert torch.equal(c.k_idx, before) and c.kv.any()


def test_append_skips_and_reports_what_is_out_of_range():
    rows, c, rope = 6, sc.empty_cache(2, "fp8", "fp8").to("cuda"), sc.rope_table(10)
    slots = torch.tensor([3, 128, -2, 5, 7, -1], dtype=torch.int32)
    pos = torch.tensor([0, 0, 0, 10, -1, 99], dtype=torch.int32)
    ws = smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), ckv=_cu(_rows(rows, 576, 1)), k_idx=_cu(_rows(rows, 128, 2)))
    assert smla.read_status(ws)[0] == 5
    for t in (c.kv, c.k_idx):
        written = t.cpu().reshape(128, -1).any(1).nonzero().flatten().tolist()
        assert written == [3]
    ws = smla.cache_append(c, _cu(slots[:1]), _cu(pos[:1]), _cu(rope), ckv=_cu(_rows(1, 576, 1)), ws=ws)
    assert smla.read_status(ws)[0] == 0


@pytest.mark.parametrize("rows,heads,h_idx,idx_dtype,inter,norm", [(1, 64, 32, "fp8", True, True), (5, 16, 4, "bf16", False, True),
                                                                   (33, 64, 64, "fp8", False, False), (130, 16, 8, "fp8", True, True),
                                                                   (70, 64, 16, "bf16", True, False)])
def test_query(rows, heads, h_idx, idx_dtype, inter, norm):
    d = 128 if idx_dtype == "fp8" else 64
    g = torch.Generator().manual_seed(rows)
    proj = torch.randn(rows, heads, 192, generator=g).to(torch.bfloat16)
    raw = _rows(rows, h_idx * d, 3, pad=16)
    w = torch.rand(rows, h_idx, generator=g) - 0.3
    iw, rope = _weights(d, 2, 1.0) if norm else None, sc.rope_table(500)
    pos = torch.randint(0, 500, (rows,), generator=g, dtype=torch.int32)
    q0 = torch.randn(rows, heads, 576, generator=g).to(torch.bfloat16)
    q = q0.cuda()
    raw_d = _strided_cuda(raw)
    _, qi, wo, ws = smla.query_prep(_cu(pos), _cu(rope), q_pe=proj.cuda()[..., 128:], q=q,
                                    q_idx_raw=raw_d.unflatten(1, (h_idx, d)), w=w.cuda(), idx_dtype=idx_dtype,
                                    idx_norm=_cu(iw), eps=EPS, w_scale=0.25, kv_interleaved=inter, idx_interleaved=not inter)
    assert smla.read_status(ws)[0] == 0
    turns = rope.numpy()[pos.numpy()][:, None]
    n64 = lambda t: t.float().double().cpu().numpy()  # noqa: E731
    assert torch.equal(q.cpu()[..., :512], q0[..., :512])
    sc.check_bf16(n64(q)[..., 512:], sc.rotate(n64(proj)[..., 128:], turns, inter))
    y = sc.rms(n64(raw).reshape(rows, h_idx, d), None if iw is None else iw.double().numpy(), EPS)
    y[..., :64] = sc.rotate(y[..., :64], turns, not inter)
    wd = w.double().numpy()
    if idx_dtype == "bf16":
        sc.check_bf16(n64(qi), y)
        np.testing.assert_allclose(n64(wo), wd * 0.25, rtol=2.0 ** -22)
    else:
        scale = sc.amax_scale(y)
        np.testing.assert_allclose(wo.cpu().double().numpy(), wd * scale * 0.25, rtol=sc.FP32)
        codes = qi.cpu().view(torch.float8_e4m3fn).float().double().numpy()
        sc.check_e4m3(codes, wo.cpu().double().numpy() / wd / 0.25, y)


def test_query_reports_positions_and_keeps_rows():
    rope = sc.rope_table(10).cuda()
    pos = torch.tensor([3, 10, -1], dtype=torch.int32, device="cuda")
    q = torch.full((3, 16, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, _, ws = smla.query_prep(pos, rope, q_pe=torch.ones(3, 16, 64, dtype=torch.bfloat16, device="cuda"), q=q)
    assert smla.read_status(ws)[0] == 5
    assert (q[1:] == 7).all() and (q[0, :, 512:] != 7).any()


# ---------------------------------------------------------------------------- attention
def _run_attention(cache, tables, lens, q_per_seq, q, shared, max_len=None, scale=sc.SM_SCALE, status=0):
    m = max(1, int(lens.max()), shared) if max_len is None else max_len
    out, lse, ws = smla.shared_prefix_fwd(cache.to("cuda"), tables.cuda(), lens.cuda(), m, shared, q_per_seq, q.cuda(), scale)
    assert smla.read_status(ws)[0] == status
    return out, lse


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("n,q,heads,shared,lens", [
    (1, 1, 64, 0, [1]),                                 # one key
    (1, 1, 16, 64, [65]),                               # a page shared, one token
    (1, 3, 64, 0, [200]),                               # nothing shared: plain causal attention
    (3, 1, 64, 128, [129, 192, 257]),                   # page borders
    (4, 2, 16, 333, [335, 400, 512, 600]),              # the shared part ends inside a page and a tile
    (5, 2, 64, 127, [0, 129, 1, 191, 300]),             # idle requests; one that is shorter than the shared part
    (9, 1, 16, 1000, [1001 + 37 * i for i in range(9)]),
    (2, 7, 64, 65, [80, 511]),
    (1, 33, 16, 100, [640]),                            # a chunk of prompt
])
def test_attention(kv_dtype, n, q, heads, shared, lens):
    c, tab, sl, qt = sc.attention_case(n, q, heads, kv_dtype, shared, lens, seed=n + q)
    out, lse = _run_attention(c, tab, sl, q, qt, shared)
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, q, qt, shared, sc.SM_SCALE), kv_dtype)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
def test_attention_long_rows(kv_dtype):
    """Keys enough to be cut into many pieces, for few rows."""
    c, tab, sl, qt = sc.attention_case(2, 1, 64, kv_dtype, 30011, [30500, 38000], seed=8)
    out, lse = _run_attention(c, tab, sl, 1, qt, 30011)
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 1, qt, 30011, sc.SM_SCALE), kv_dtype)


def test_attention_peaked_and_rising_logits():
    """Logits of up to some hundreds whose running maximum keeps rising."""
    c, tab, sl, qt = sc.attention_case(2, 2, 16, "bf16", 700, [900, 1300], seed=4, q_std=12.0)
    c.kv *= torch.linspace(0.1, 3.0, c.kv.shape[0])[:, None, None].to(torch.bfloat16)
    out, lse = _run_attention(c, tab, sl, 2, qt, 700)
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 2, qt, 700, sc.SM_SCALE), "bf16")


def test_attention_many_requests():
    rng = np.random.default_rng(3)
    lens = (150 + rng.integers(0, 120, 130)).tolist()
    c, tab, sl, qt = sc.attention_case(130, 1, 16, "bf16", 150, lens, seed=5)
    out, lse = _run_attention(c, tab, sl, 1, qt, 150)
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 1, qt, 150, sc.SM_SCALE), "bf16")


def test_attention_new_tokens_nan_stays_with_those_that_see_it():
    """The last new token's key is NaN: the tokens before it do not see it."""
    c, tab, sl, qt = sc.attention_case(2, 4, 16, "bf16", 100, [260, 131], seed=6)
    last = [(tab[b, (int(sl[b]) - 1) // 64], (int(sl[b]) - 1) % 64) for b in range(2)]
    ref = sc.attention_reference(c, tab, sl, 4, qt, 100, sc.SM_SCALE)
    for p, s in last:
        c.kv[p, s] = float("nan")
    out, lse = _run_attention(c, tab, sl, 4, qt, 100)
    seen = [r for r in range(8) if r % 4 != 3]
    sc.check_attention(out[seen], lse[seen], tuple(a[seen] for a in ref), "bf16")
    assert out[3::4].isnan().all() and lse[3::4].isnan().all()


@pytest.mark.parametrize("scale", [-0.04, 0.0, 1e-6, 0.5])
def test_attention_softmax_scales(scale):
    c, tab, sl, qt = sc.attention_case(2, 2, 16, "bf16", 130, [300, 211], seed=14)
    out, lse = _run_attention(c, tab, sl, 2, qt, 130, scale=scale)
    ref = sc.attention_reference(c, tab, sl, 2, qt, 130, scale)
    sc.check_attention(out, lse, ref[:3] + (np.abs(ref[3]),), "bf16")


@pytest.mark.parametrize("factor", [1e-25, 1e-12, 1e12])
def test_attention_per_token_scales_of_any_size(factor):
    """Scales far from one, and some that are zero (a row of zeros)."""
    c, tab, sl, qt = sc.attention_case(2, 1, 16, "fp8", 200, [420, 333], seed=15)
    live = torch.isfinite(c.kv_scale)
    c.kv_scale[live] *= factor * (1 + torch.arange(c.kv_scale.numel()).view_as(c.kv_scale) % 7)[live]
    c.kv_scale[torch.logical_and(live, torch.arange(64)[None] % 5 == 0)] = 0.0
    scale = sc.SM_SCALE / max(factor, 1.0)
    out, lse = _run_attention(c, tab, sl, 1, qt, 200, scale=scale)
    sc.check_attention(out.float() / 1.0, lse, sc.attention_reference(c, tab, sl, 1, qt, 200, scale), "fp8")


def test_attention_nan_scale_reaches_only_those_that_see_it():
    c, tab, sl, qt = sc.attention_case(1, 3, 16, "fp8", 0, [150], seed=16)
    ref = sc.attention_reference(c, tab, sl, 3, qt, 0, sc.SM_SCALE)
    c.kv_scale[tab[0, 149 // 64], 149 % 64] = float("nan")
    out, lse = _run_attention(c, tab, sl, 3, qt, 0)
    sc.check_attention(out[:2], lse[:2], tuple(a[:2] for a in ref), "fp8")
    assert out[2].isnan().all() and lse[2].isnan().all()


@pytest.mark.parametrize("kv_dtype,what", [("fp8_ds_mla", "query"), ("fp8_ds_mla", "row")])
def test_attention_reports_values_outside_f16(kv_dtype, what):
    c, tab, sl, qt = sc.attention_case(1, 1, 16, kv_dtype, 0, [100], seed=17)
    if what == "query":
        qt[0, 3, 5] = 1e5
    else:
        c.kv[tab[0, 0], 7, 512:516] = torch.tensor([1e4], dtype=torch.float32).view(torch.uint8)
        c.kv[tab[0, 0], 7, 0] = 0x7E  # 448
    _, _, ws = smla.shared_prefix_fwd(c.to("cuda"), tab.cuda(), sl.cuda(), 100, 0, 1, qt.cuda(), sc.SM_SCALE)
    assert smla.read_status(ws)[0] == 2


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("q", [1, 2])
def test_attention_bad_page_is_skipped_and_reported(kv_dtype, q):
    for bad in ((0, 1), (1, 6)):  # in the shared part; in a request's own
        c, tab, sl, qt = sc.attention_case(2, q, 64, kv_dtype, 256, [500, 470], seed=7)
        tab[bad] = 10 ** 6 if q == 1 else -3
        out, lse = _run_attention(c, tab, sl, q, qt, 256, status=5)
        sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, q, qt, 256, sc.SM_SCALE), kv_dtype)


def test_attention_length_above_its_bound_is_reported():
    c, tab, sl, qt = sc.attention_case(2, 1, 16, "bf16", 64, [200, 150], seed=9)
    ref = sc.attention_reference(c, tab, torch.tensor([180, 150]), 1, qt, 64, sc.SM_SCALE)
    out, lse = _run_attention(c, tab, sl, 1, qt, 64, max_len=180, status=5)
    sc.check_attention(out, lse, ref, "bf16")


def test_attention_repeats_on_another_stream_and_in_a_graph():
    """The same call twice, on a side stream and replayed from a graph: the same bits; nothing outside the outputs is written."""
    c, tab, sl, qt = sc.attention_case(3, 2, 64, "bf16", 200, [260, 410, 777], seed=10)
    c, tab, sl, qt = c.to("cuda"), tab.cuda(), sl.cuda(), qt.cuda()
    ws = smla.workspace(smla.shared_prefix_workspace_bytes(3, 777, 200, 2, 64))
    raw = torch.full((6 * 64 * 512 + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = raw[2048:-2048].view(6, 64, 512)
    call = lambda: smla.shared_prefix_fwd(c, tab, sl, 777, 200, 2, qt, sc.SM_SCALE, out=out, lse=lse, ws=ws)  # noqa: E731
    lse = torch.empty(6, 64, device="cuda")
    call()
    first, flse = out.clone(), lse.clone()
    assert (raw[:2048] == 3).all() and (raw[-2048:] == 3).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, flse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, flse)


def test_attention_agrees_with_sparse_over_all_keys():
    """Every key selected: the sparse attention over all positions gives the same rows."""
    n, q, heads, shared, lens = 2, 2, 64, 192, [700, 512]
    c, tab, sl, qt = sc.attention_case(n, q, heads, "bf16", shared, lens, seed=12)
    out, lse = _run_attention(c, tab, sl, q, qt, shared)
    tab[1, :shared // 64] = tab[0, :shared // 64]
    idx = torch.arange(704, dtype=torch.int32).expand(n * q, 704).contiguous()
    so, sl_, _ = smla.sparse_mla_fwd(c.to("cuda"), tab.cuda(), qt.cuda(), idx.cuda(), sc.SM_SCALE, seq_lens=sl.cuda(), q_per_seq=q)
    ref = sc.attention_reference(c, tab, sl, q, qt, shared, sc.SM_SCALE)
    sc.check_attention(out, lse, ref, "bf16")
    sc.check_attention(so, sl_, ref, "bf16")


def test_many_rows_report_bad_rows_too():
    """Past the size up to which one block reports: the same skips, the same status."""
    rows, c, rope = 5000, sc.empty_cache(80, "bf16", "fp8").to("cuda"), sc.rope_table(10)
    slots = torch.arange(rows, dtype=torch.int32)
    slots[4321] = 10 ** 6
    pos = torch.zeros(rows, dtype=torch.int32)
    ws = smla.cache_append(c, _cu(slots), _cu(pos), _cu(rope), ckv=_cu(_rows(rows, 576, 1)), k_idx=_cu(_rows(rows, 128, 2)))
    assert smla.read_status(ws)[0] == 5
    assert c.kv.cpu().reshape(80 * 64, -1).any(1).sum() == rows - 1
    pos[77] = 10
    q = torch.zeros(rows, 16, 576, dtype=torch.bfloat16, device="cuda")
    pe = torch.ones(rows, 16, 64, dtype=torch.bfloat16, device="cuda")
    _, _, _, ws = smla.query_prep(_cu(pos), _cu(rope), q_pe=pe, q=q)
    assert smla.read_status(ws)[0] == 5
    assert q.any(2).all(1).sum() == rows - 1
    pos[77] = 9
    _, _, _, ws = smla.query_prep(_cu(pos), _cu(rope), q_pe=pe, q=q, ws=ws)
    assert smla.read_status(ws)[0] == 0 and q.any(2).all()
