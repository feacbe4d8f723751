"""The serving operators where their contracts end. References: serve_common."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import serve_bounds as sb
import serve_common as sc

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "fp8", "fp8_ds_mla"]


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


# ---------------------------------------------------------------------------- e4m3 codes
def _codes(x):
    """scale and codes of the last axis in fp32 as the header defines them: amax / 448 (at least 2^-126), x / scale to nearest even."""
    top = np.abs(x).max(-1)
    scale = np.where(top > 0, np.maximum(top / np.float32(448), np.float32(2.0 ** -126)), np.float32(1)).astype(np.float32)
    return scale, torch.from_numpy((x / scale[..., None]).astype(np.float32)).to(torch.float8_e4m3fn).float().numpy()


def _spread(*shape, seed):
    """bf16 values whose rows have magnitudes from 2^-110 to 2^110."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-110, 111, shape[:-1] + (1,), generator=g).float())
    x.view(-1, shape[-1])[::5] = torch.randn(x.view(-1, shape[-1])[::5].shape, generator=g)  # every fifth row about one
    return x.to(torch.bfloat16)


def _unturned(rows):
    """(positions, table): position 0 turns by no angle, so that values reach their codes as they are."""
    return torch.zeros(rows, dtype=torch.int32, device="cuda"), sc.rope_table(1).cuda()


@pytest.mark.parametrize("kv_dtype", ["fp8", "fp8_ds_mla"])
def test_append_codes_are_the_rounded_quotients(kv_dtype):
    rows = 4999
    ckv, kr = _spread(rows, 576, seed=1), _spread(rows, 128, seed=2)
    c = sc.empty_cache(rows // 64 + 1, kv_dtype, "fp8").to("cuda")
    pos, rope = _unturned(rows)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    ws = smla.cache_append(c, slots, pos, rope, ckv=ckv.cuda(), k_idx=kr.cuda())
    assert smla.read_status(ws)[0] == 0
    f8 = lambda b: b.contiguous().view(torch.float8_e4m3fn).float().numpy()  # noqa: E731
    kv, x = c.kv.cpu().reshape(-1, c.kv.shape[-1])[:rows], ckv.float().numpy()
    if kv_dtype == "fp8":
        got_scale, got = c.kv_scale.cpu().numpy().reshape(-1)[:rows], f8(kv)
    else:
        x = x[:, :512].reshape(rows, 4, 128)
        got_scale, got = kv[:, 512:528].contiguous().view(torch.float32).numpy(), f8(kv[:, :512]).reshape(rows, 4, 128)
    scale, codes = _codes(x)
    assert np.array_equal(got_scale, scale)
    assert np.array_equal(got, codes)
    scale, codes = _codes(kr.float().numpy())
    assert np.array_equal(c.k_idx_scale.cpu().numpy().reshape(-1)[:rows], scale)
    assert np.array_equal(f8(c.k_idx.cpu().reshape(-1, 128)[:rows]), codes)


@pytest.mark.parametrize("rows", [300, 4500])  # (4,500: the status word is cleared by a launch of its own)
def test_query_codes_are_the_rounded_quotients(rows):
    raw = _spread(rows, 8, 128, seed=rows)
    pos, rope = _unturned(rows)
    w = torch.ones(rows, 8, device="cuda")
    _, qi, wo, ws = smla.query_prep(pos, rope, q_idx_raw=raw.cuda(), w=w)
    assert smla.read_status(ws)[0] == 0
    scale, codes = _codes(raw.float().numpy())
    assert np.array_equal(wo.cpu().numpy(), scale)
    assert np.array_equal(qi.cpu().view(torch.float8_e4m3fn).float().numpy(), codes)


def test_append_codes_of_the_ends_of_fp32():
    """An infinite amax, NaN, zeros, and rows whose scale would fall below 2^-126."""
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(6, 128, dtype=torch.bfloat16)  # (values from 64 on are not rotated)
    x[0, 64:68] = torch.tensor([inf, -inf, 3.0, -3e38])
    x[1, 64:67] = torch.tensor([nan, 2.0, -448.0])
    x[2, 64:68] = torch.tensor([2.0 ** -118, -3 * 2.0 ** -121, 2.0 ** -126, 2.0 ** -130])
    x[3, 64:67] = torch.tensor([2.0 ** -126, -(2.0 ** -128), 2.0 ** -133])
    x[4, 64:67] = torch.tensor([3.3e38, -1e38, 1e36])
    c = sc.empty_cache(1, "bf16", "fp8").to("cuda")
    pos, rope = _unturned(6)
    smla.cache_append(c, torch.arange(6, dtype=torch.int32, device="cuda"), pos, rope, k_idx=x.cuda())
    scale = c.k_idx_scale.cpu().numpy()[0, :6]
    got = c.k_idx.cpu()[0, :6].view(torch.float8_e4m3fn).float().numpy()
    with np.errstate(invalid="ignore"):
        want_scale, want = _codes(np.nan_to_num(x.float().numpy(), nan=0.0, posinf=np.inf, neginf=-np.inf))
    want[0, 64:68] = [nan, nan, 0, 0]  # infinity by infinity; finite by infinity
    want[1, 64] = nan
    assert np.array_equal(scale, want_scale) and np.isinf(scale[0]) and scale[3] == 2.0 ** -126 and scale[5] == 1
    np.testing.assert_array_equal(got, want)


# ---------------------------------------------------------------------------- memory that no row sees
def _attend(c, tab, sl, q, qt, shared, max_len=None, scale=sc.SM_SCALE):
    m = max(1, int(sl.max()), shared) if max_len is None else max_len
    out, lse, ws = smla.shared_prefix_fwd(c.to("cuda"), tab.cuda(), sl.cuda(), m, shared, q, qt.cuda(), scale)
    return out, lse, smla.read_status(ws)[0]


def _huge(c, dead):
    """Tile-scaled rows whose values are finite and far outside f16's range."""
    c.kv[dead] = torch.cat([torch.full((512,), 0x7E, dtype=torch.uint8), torch.full((4,), 1e30).view(torch.uint8),
                            torch.full((64,), 1e30, dtype=torch.bfloat16).view(torch.uint8)])


@pytest.mark.parametrize("n,q,heads,shared,lens", [
    (1, 1, 64, 0, [100]),                   # past the length
    (1, 5, 64, 0, [77]),
    (2, 1, 16, 130, [200, 333]),            # and before the border of the second request's page (one row block)
    (3, 2, 64, 200, [260, 410, 777]),       # the shared part's copy (three row blocks)
])
def test_attention_unseen_values_outside_f16_are_not_reported(n, q, heads, shared, lens):
    c, tab, sl, qt = sc.attention_case(n, q, heads, "fp8_ds_mla", shared, lens, seed=n + 20)
    _huge(c, (c.kv == 0xFF).all(-1))
    ref = sc.attention_reference(c, tab, sl, q, qt, shared, sc.SM_SCALE)
    out, lse, status = _attend(c, tab, sl, q, qt, shared)
    assert status == 0
    sc.check_attention(out, lse, ref, "fp8_ds_mla")


@pytest.mark.parametrize("q,heads", [(1, 16), (2, 64)])
def test_attention_shared_values_past_every_length_are_not_reported(q, heads):
    """All requests end before the shared part does."""
    c, tab, sl, qt = sc.attention_case(3, q, heads, "fp8_ds_mla", 333, [100, 90, 70], seed=24)
    for s in range(100, 333):
        _huge(c, (tab[0, s // 64], s % 64))
    ref = sc.attention_reference(c, tab, sl, q, qt, 333, sc.SM_SCALE)
    out, lse, status = _attend(c, tab, sl, q, qt, 333)
    assert status == 0
    sc.check_attention(out, lse, ref, "fp8_ds_mla")
    _huge(c, (tab[0, 1], 99 % 64))  # the last one that a row sees
    assert _attend(c, tab, sl, q, qt, 333)[2] == 2


@pytest.mark.parametrize("shared", [0, 130])
def test_attention_queries_that_see_nothing_are_not_reported(shared):
    c, tab, sl, qt = sc.attention_case(3, 2, 64, "fp8_ds_mla", shared, [0, 180, 1], seed=25)
    qt[0:2], qt[4] = 1e30, -1e30  # an idle request, and a token before the first key
    out, lse, status = _attend(c, tab, sl, 2, qt, shared)
    assert status == 0
    qt[0:2], qt[4] = 0, 0
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 2, qt, shared, sc.SM_SCALE), "fp8_ds_mla")


# ---------------------------------------------------------------------------- idle requests
@pytest.mark.parametrize("kv_dtype", FORMATS)
@pytest.mark.parametrize("n,q,heads", [(2, 1, 16), (5, 2, 64)])  # one and several row blocks
def test_attention_of_an_idle_batch_looks_at_no_page(kv_dtype, n, q, heads):
    c, tab, sl, qt = sc.attention_case(n, q, heads, kv_dtype, 200, [0] * n, seed=26)
    tab[:] = -1
    out, lse, status = _attend(c, tab, sl, q, qt, 200, max_len=256)
    assert status == 0 and (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kv_dtype", FORMATS)
@pytest.mark.parametrize("n,q,heads", [(3, 1, 16), (6, 2, 64)])
def test_attention_pages_past_every_length_need_not_exist(kv_dtype, n, q, heads):
    lens = [130, 70, 0, 5, 129, 0][:n]
    c, tab, sl, qt = sc.attention_case(n, q, heads, kv_dtype, 700, lens, seed=27)
    tab[:, 3:] = -1
    out, lse, status = _attend(c, tab, sl, q, qt, 700)
    assert status == 0
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, q, qt, 700, sc.SM_SCALE), kv_dtype)
    tab[0, 2] = -1  # keys 128 and 129: seen by request 0 (and 4)
    out, lse, status = _attend(c, tab, sl, q, qt, 700)
    assert status == 5
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, q, qt, 700, sc.SM_SCALE), kv_dtype)


@pytest.mark.parametrize("kv_dtype", FORMATS)
def test_attention_idle_requests_among_others(kv_dtype):
    """Row blocks of idle requests between others, the first among them: its table lists the prompt all the same."""
    lens = [0, 0, 0, 900, 0, 650, 0, 0, 0, 0, 701, 0, 40, 0]
    c, tab, sl, qt = sc.attention_case(14, 1, 64, kv_dtype, 640, lens, seed=28)
    out, lse, status = _attend(c, tab, sl, 1, qt, 640)
    assert status == 0
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 1, qt, 640, sc.SM_SCALE), kv_dtype)


@pytest.mark.parametrize("kv_dtype", FORMATS)
def test_attention_more_row_blocks_than_the_table_of_ends_holds(kv_dtype):
    """1,040 requests of 64 heads: 520 row blocks share 130 keys, two of them an end; whole blocks of them are idle."""
    rng = np.random.default_rng(29)
    lens = np.where(np.arange(1040) % 37 < 9, rng.integers(0, 190, 1040), 0).tolist()
    c, tab, sl, qt = sc.attention_case(1040, 1, 64, kv_dtype, 130, lens, seed=29)
    out, lse, status = _attend(c, tab, sl, 1, qt, 130)
    assert status == 0
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 1, qt, 130, sc.SM_SCALE), kv_dtype)


# ---------------------------------------------------------------------------- nothing shared, many segments
def _sample(tab, sl, q, qt, rows):
    """Rows of a batch as requests of one token each (row 0 first: its table holds the shared part)."""
    rows = [0] + sorted(rows)
    b = [r // q for r in rows]
    lens = [max(0, int(sl[r // q]) - q + r % q + 1) for r in rows]
    return rows, tab[b], torch.tensor(lens, dtype=torch.int32), qt[rows]


@pytest.mark.parametrize("kv_dtype", FORMATS)
@pytest.mark.parametrize("n,q,heads,longest", [
    (1, 1101, 64, 1500),  # a chunk of prompt: 551 segments of up to 12 tiles, most of them uncut
    (1, 700, 16, 5003),   # 88 segments of 34 to 40 tiles: a pair walks one and a bit
    (90, 3, 64, 700),     # 180 segments, two a request
    (601, 1, 64, 150),    # more segments than threads
])
def test_attention_nothing_shared_many_segments(kv_dtype, n, q, heads, longest):
    rng = np.random.default_rng(n)
    lens = [longest] if n == 1 else rng.integers(0, longest + 1, n).tolist()
    c, tab, sl, qt = sc.attention_case(n, q, heads, kv_dtype, 0, lens, seed=30)
    need = smla.shared_prefix_workspace_bytes(n, longest, 0, q, heads, kv_dtype)
    raw = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse, ws = smla.shared_prefix_fwd(c.to("cuda"), tab.cuda(), sl.cuda(), longest, 0, q, qt.cuda(), sc.SM_SCALE, ws=raw[:need])
    assert smla.read_status(ws)[0] == 0 and (raw[need:] == 0xA5).all()
    assert out.isfinite().all()
    rows, t, l, x = _sample(tab, sl, q, qt, rng.choice(n * q, 60, replace=False).tolist())
    sc.check_attention(out[rows], lse[rows], sc.attention_reference(c, t, l, 1, x, 0, sc.SM_SCALE), kv_dtype)


# ---------------------------------------------------------------------------- long rows, small values, other inputs
@pytest.mark.parametrize("kv_dtype", FORMATS)
def test_attention_long_rows_as_a_whole(kv_dtype):
    """Bounds that a lost tile of keys does not pass (one row block's keys in pieces; the copy of shared rows)."""
    for n, q, shared, lens in ((1, 1, 0, [38000]), (3, 2, 30011, [38000, 9000, 30200])):
        c, tab, sl, qt = sc.attention_case(n, q, 64, kv_dtype, shared, lens, seed=31)
        out, lse, status = _attend(c, tab, sl, q, qt, shared)
        assert status == 0
        ro, rl, _, _ = sc.attention_reference(c, tab, sl, q, qt, shared, sc.SM_SCALE)
        sb.check_rows(out.double().cpu().numpy(), lse.double().cpu().numpy(), ro, rl)


@pytest.mark.parametrize("factor", [1e-3, 1e-5, 1e-7, 1e-9])
def test_attention_small_tile_scaled_values(factor):
    """Values below f16's normals (2^-14) are held to 2^-25: the results' error grows by that, and a logit's by
    that much of each |q|."""
    c, tab, sl, qt = sc.attention_case(2, 1, 16, "fp8_ds_mla", 200, [420, 333], seed=32)
    live = ~(c.kv == 0xFF).all(-1)
    scales = c.kv[..., 512:528].contiguous().view(torch.float32)
    scales[live] *= factor
    c.kv[..., 512:528] = scales.view(torch.uint8)
    out, lse, status = _attend(c, tab, sl, 1, qt, 200)
    assert status == 0
    ro, rl, mag, top = sc.attention_reference(c, tab, sl, 1, qt, 200, sc.SM_SCALE)
    delta = top * (576 * 2.0 ** -24 + 2.0 ** -11) + 2.0 ** -18 + 2.0 ** -25 * sc.SM_SCALE * qt.double().abs().sum(-1).numpy()
    rel = (2.0 ** -10 + 2.0 ** -14 + 2 * delta)[..., None]
    bound = rel * mag + 2.0 ** -25 * (1 + rel)
    assert (np.abs(out.double().cpu().numpy() - ro) <= bound + 2.0 ** -8 * (np.abs(ro) + bound)).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= delta + 2.0 ** -20 * np.abs(rl)).all()


@pytest.mark.parametrize("kv_dtype", FORMATS)
@pytest.mark.parametrize("n", [2, 5])
def test_attention_queries_on_a_16_byte_boundary(kv_dtype, n):
    c, tab, sl, qt = sc.attention_case(n, 2, 64, kv_dtype, 130, [300, 411, 129, 0, 257][:n], seed=33)
    base = torch.empty(qt.numel() + 8, dtype=torch.bfloat16, device="cuda")
    q = base[8:].view(qt.shape)
    q.copy_(qt)
    assert q.data_ptr() % 32 == 16
    m = int(sl.max())
    out, lse, ws = smla.shared_prefix_fwd(c.to("cuda"), tab.cuda(), sl.cuda(), m, 130, 2, q, sc.SM_SCALE)
    assert smla.read_status(ws)[0] == 0
    sc.check_attention(out, lse, sc.attention_reference(c, tab, sl, 2, qt, 130, sc.SM_SCALE), kv_dtype)


@pytest.mark.parametrize("kv_dtype", ["fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("n", [1, 4])
def test_attention_negative_scale_of_fp8_rows(kv_dtype, n):
    c, tab, sl, qt = sc.attention_case(n, 2, 64, kv_dtype, 130, [300, 211, 140, 500][:n], seed=34)
    out, lse, status = _attend(c, tab, sl, 2, qt, 130, scale=-0.04)
    assert status == 0
    ref = sc.attention_reference(c, tab, sl, 2, qt, 130, -0.04)
    sc.check_attention(out, lse, ref[:3] + (np.abs(ref[3]),), kv_dtype)


@pytest.mark.parametrize("kv_dtype", ["fp8", "fp8_ds_mla"])
def test_attention_copy_of_shared_rows_on_streams_and_in_graphs(kv_dtype):
    """The 16-bit copy is made anew by every call: in a workspace full of NaN, after another prompt, on a side stream
    and by a replayed graph, the same bits."""
    a, b = (sc.attention_case(4, 2, 64, kv_dtype, 450, [600, 451, 777, 500], seed=s) for s in (35, 36))
    ref = sc.attention_reference(*a[:3], 2, a[3], 450, sc.SM_SCALE)
    (ca, ta, la, qa), (cb, tb, lb, qb) = ((c.to("cuda"), t.cuda(), sl.cuda(), q.cuda()) for c, t, sl, q in (a, b))
    ws = smla.workspace(smla.shared_prefix_workspace_bytes(4, 777, 450, 2, 64, kv_dtype)).fill_(0xFF)
    out, lse = torch.empty(8, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 64, device="cuda")
    call = lambda c, t, sl, q: smla.shared_prefix_fwd(c, t, sl, 777, 450, 2, q, sc.SM_SCALE, out=out, lse=lse, ws=ws)  # noqa: E731
    call(ca, ta, la, qa)
    assert smla.read_status(ws)[0] == 0
    sc.check_attention(out, lse, ref, kv_dtype)
    first, flse = out.clone(), lse.clone()
    same = lambda: torch.equal(out, first) and torch.equal(lse, flse)  # noqa: E731
    call(cb, tb, lb, qb)
    assert not same()
    call(ca, ta, la, qa)
    assert same()
    call(cb, tb, lb, qb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ca, ta, la, qa)
    side.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(cb, tb, lb, qb)
        call(ca, ta, la, qa)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert same()


@pytest.mark.parametrize("kv_dtype", FORMATS)
def test_attention_many_rows_on_a_shared_prompt(kv_dtype):
    """38,464 rows of 601 requests: each block of the joining kernel takes all of its rows' values."""
    rng = np.random.default_rng(37)
    lens = (200 + rng.integers(0, 70, 601)).tolist()
    c, tab, sl, qt = sc.attention_case(601, 1, 64, kv_dtype, 200, lens, seed=37)
    out, lse, status = _attend(c, tab, sl, 1, qt, 200)
    assert status == 0 and out.isfinite().all()
    rows, t, l, x = _sample(tab, sl, 1, qt, rng.choice(601, 80, replace=False).tolist())
    sc.check_attention(out[rows], lse[rows], sc.attention_reference(c, t, l, 1, x, 200, sc.SM_SCALE), kv_dtype)


# ---------------------------------------------------------------------------- tables
def _tables(ctx, new, tables, free, max_new):
    i = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    tab = i(tables)
    seq, cu, pos, slots, own, used, ws = smla.build_tables(i(ctx), i(new), tab, i(free), max_new)
    return seq.tolist(), slots.tolist(), tab.tolist(), int(used), smla.read_status(ws)[0]


@pytest.mark.parametrize("bad", [-1, -7, 1 << 25, 2 ** 31 - 1])
def test_tables_report_unusable_ids_of_the_free_list(bad):
    # 64 tokens and 70 more: pages free[0], free[1]; an empty request with 3: free[2]
    for at in range(3):
        free = [10, 11, 12, -1]  # (the last one is not taken)
        free[at] = bad
        seq, slots, tab, used, status = _tables([64, 0], [70, 3], [[5, -1, -1], [-1, -1, -1]], free, 73)
        assert status == 5 and used == 3 and seq == [134, 3]
        page = lambda i, rows: [-1] * rows if i == at else [free[i] * 64 + r for r in range(rows)]  # noqa: E731
        assert slots == page(0, 64) + page(1, 6) + page(2, 3)
        assert tab == [[5, free[0], free[1]], [free[2], -1, -1]]
    assert _tables([64, 0], [70, 3], [[5, -1, -1], [-1, -1, -1]], [10, 11, 12, -1], 73)[4] == 0


def test_tables_report_an_unusable_id_far_down_the_free_list():
    free = np.arange(5000)
    n, lens = 2000, [64] * 2000
    assert _tables([0] * n, lens, [[-1]] * n, free, 64 * n)[4] == 0
    free[1999] = -1
    seq, slots, _, used, status = _tables([0] * n, lens, [[-1]] * n, free, 64 * n)
    assert status == 5 and used == 2000 and slots[-65:] == [1998 * 64 + 63] + [-1] * 64


@pytest.mark.parametrize("bad", [-1, 1 << 25])
def test_tables_report_an_unusable_page_in_use(bad):
    seq, slots, _, used, status = _tables([70], [60], [[5, bad, -1]], [9], 60)
    assert status == 5 and slots == [-1] * 58 + [9 * 64, 9 * 64 + 1] and seq == [130] and used == 1


def test_tables_lengths_next_to_the_end_of_int32():
    """Positions and page numbers stay in 32 bits: 2^31 - 64 tokens are the most that a request can have."""
    width, last = 1 << 25, 2 ** 31 - 64
    tab = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    tab[0, last // 64 - 1] = 7
    free = torch.tensor([9], dtype=torch.int32, device="cuda")
    i = lambda a: torch.tensor([a], dtype=torch.int32, device="cuda")  # noqa: E731
    seq, cu, pos, slots, _, used, ws = smla.build_tables(i(last - 3), i(3), tab, free, 4)
    assert smla.read_status(ws)[0] == 0 and int(seq) == last and int(used) == 0
    assert pos.tolist() == [last - 3, last - 2, last - 1, -1] and slots.tolist() == [7 * 64 + 61, 7 * 64 + 62, 7 * 64 + 63, -1]
    for ctx, new in ((last - 3, 4), (last, 1), (last + 50, 1), (2 ** 31 - 1, 1), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)):
        seq, cu, pos, slots, _, used, ws = smla.build_tables(i(ctx), i(new), tab, free, 4)
        assert smla.read_status(ws)[0] == 5 and int(seq) == 0 and cu.tolist() == [0, 0] and int(used) == 0
        assert slots.tolist() == [-1] * 4 and (tab == -1).sum() == width - 1


# ---------------------------------------------------------------------------- padding
def test_query_skips_the_padding_of_the_tables():
    """Rows past a batch's own have position -1 (build_tables): nothing is written, nothing reported."""
    rope = sc.rope_table(100).cuda()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    _, _, pos, slots, _, _, ws = smla.build_tables(i([3, 0]), i([2, 1]), i([[4], [-1]]), i([7]), 8)
    assert smla.read_status(ws)[0] == 0 and pos.tolist() == [3, 4, 0] + [-1] * 5
    for rows in (8, 5000):  # (past 4,096 rows the warps report)
        p = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        p[:8] = pos
        q = torch.full((rows, 16, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        qi = torch.full((rows, 4, 128), 9, dtype=torch.uint8, device="cuda")
        wo = torch.full((rows, 4), 5.0, device="cuda")
        _, _, _, ws = smla.query_prep(p, rope, q_pe=torch.ones(rows, 16, 64, dtype=torch.bfloat16, device="cuda"), q=q, q_idx=qi, w_out=wo,
                                      q_idx_raw=torch.ones(rows, 4, 128, dtype=torch.bfloat16, device="cuda"), w=torch.ones(rows, 4, device="cuda"))
        assert smla.read_status(ws)[0] == 0
        assert (q[3:] == 7).all() and (qi[3:] == 9).all() and (wo[3:] == 5).all()
        assert (q[:3, :, 512:] != 7).any(-1).all() and (wo[:3] != 5).all()
        for bad in (-2, 100):
            p[5] = bad
            _, _, _, ws = smla.query_prep(p, rope, q_pe=torch.ones(rows, 16, 64, dtype=torch.bfloat16, device="cuda"), q=q)
            assert smla.read_status(ws)[0] == 5
