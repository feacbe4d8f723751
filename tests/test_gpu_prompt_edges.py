"""Calls at the edges of what include/smla_prompt.h allows, on the GPU."""
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import prompt_common as pc
import prompt_tiles as pt
from test_gpu_prompt import _bf16_rows, _filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


# ---------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("lead", [16, 32, 48])
@pytest.mark.parametrize("ql,kl", [([2, 1, 5], [9000, 3, 17000]), ([300], [5000]), ([70, 9], [90, 20])])
def test_prompt_workspace_on_any_16_byte_boundary(lead, ql, kl):
    """Cut keys (partial results in the workspace), uncut ones, a call without a plan: the bits that the allocator's own
    boundary gives, and nothing written behind the size that the call asks for."""
    q, k, v, pe, cq, ck = (t.cuda() for t in pc.prompt_case(ql, kl, 4, 4, 192, True, seed=50))
    need = smla.prompt_workspace_bytes(sum(ql), sum(kl), len(ql), 4, 4)
    call = lambda ws: smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, ws=ws)  # noqa: E731
    out, lse, _ = call(smla.workspace(need))
    raw = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws = raw[lead:lead + need]
    assert ws.data_ptr() % 64 == lead % 64
    got, glse, _ = call(ws)
    assert smla.read_status(ws)[0] == 0
    assert torch.equal(got, out) and torch.equal(glse, lse)
    assert (raw[:lead] == 171).all() and (raw[lead + need:] == 171).all()


# ---------------------------------------------------------------------------- values that are not finite
def _levels(nk, low, size=128, even=True, first=None):
    """Logits by key: `low` in every other tile of 128 keys, or in the keys before `first`; 0 elsewhere."""
    j = torch.arange(nk)
    hit = j < first if first is not None else ((j // size) % 2 == 0) == even
    return torch.where(hit, low, 0.0)


def _level_case(nq, level, seed):
    """One head whose logits with a scale of 1 are `level`, whatever the query; random values."""
    g = torch.Generator().manual_seed(seed)
    nk = level.numel()
    q, k = torch.zeros(nq, 1, 128, dtype=torch.bfloat16), torch.zeros(nk, 1, 128, dtype=torch.bfloat16)
    q[:, 0, 0], k[:, 0, 0] = 1.0, level.to(torch.bfloat16)
    return q.cuda(), k.cuda(), torch.randn(nk, 1, 128, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("low", [-300.0, -float("inf")])
@pytest.mark.parametrize("nq,nk,even,first", [
    (100, 512, True, None), (100, 512, False, None), (1, 1100, True, None),   # key tiles in two halves of the pipeline
    (2, 30000, True, 15000), (2, 30000, True, 29000), (200, 20000, False, None),  # cut keys
    (300, 512, True, None), (300, 512, True, 200)])                           # two row tiles
def test_prompt_values_whose_weight_vanishes(nq, nk, even, first, low):
    """A NaN or an infinity of V at a key that every row sees reaches every row, however small the key's probability."""
    level = _levels(nk, low, even=even, first=first)
    q, k, v = _level_case(nq, level, 70)
    odd = int((level < 0).nonzero()[0])
    v[odd, 0, 3], v[odd + 1, 0, 7], v[odd + 2, 0, 9] = float("nan"), float("inf"), -float("inf")
    out, lse, ws = smla.prompt_fwd(q, k, v.cuda(), pc.cu([nq], "cuda"), pc.cu([nk], "cuda"), 1.0, causal=False)
    assert smla.read_status(ws)[0] == 0
    live = level == 0
    assert out[:, 0, 3].isnan().all()
    assert not torch.isfinite(out[:, 0, [7, 9]]).any()
    rest = [c for c in range(128) if c not in (3, 7, 9)]
    want = v[live, 0].double().mean(0)[rest]
    mag = v[live, 0].double().abs().mean(0)[rest]
    # equal probabilities: exact but for the sums (2^-23 a key of the mean magnitude) and bf16
    assert ((out[:, 0, rest].double().cpu() - want).abs() <= pc.BF16 * want.abs() + 2 * pc.FP32 * nk * mag).all()
    assert ((lse.cpu() - float(live.sum().double().log())).abs() <= 2.0 ** -16).all()


@pytest.mark.parametrize("nq,nk", [(100, 300), (3, 20000)])
def test_prompt_joined_values_whose_weight_vanishes(nq, nk):
    """The earlier result's values too, and this call's beside an earlier result that outweighs them; -inf adds nothing."""
    q, k, v = _level_case(nq, torch.zeros(nk), 71)
    po, pl = torch.randn(nq, 1, 128, generator=torch.Generator().manual_seed(72)), torch.full((nq, 1), -400.0)
    po[0, 0, 5], pl[1, 0], pl[2, 0] = float("nan"), 500.0, -float("inf")
    po[2] = float("nan")
    v[40, 0, 9] = float("nan")
    out, lse, ws = smla.prompt_fwd(q, k, v.cuda(), pc.cu([nq], "cuda"), pc.cu([nk], "cuda"), 1.0, causal=False, prev_out=po.cuda(), prev_lse=pl.cuda(),
                                   out_dtype=torch.float32)
    assert smla.read_status(ws)[0] == 0
    bad = out.isnan().cpu()[:, 0]
    want = torch.zeros_like(bad)
    want[:, 9] = True
    want[0, 5] = True
    assert torch.equal(bad, want)
    rest = ~want[1]
    assert torch.equal(out[1, 0].cpu()[rest], po[1, 0][rest]) and lse[1, 0] == 500.0


def test_prompt_rows_whose_logits_are_all_minus_infinity():
    """They are as rows that see nothing, whole or cut, alone or joined, whatever V holds."""
    for nq, nk, odd in ((100, 300, 290), (300, 300, 5), (300, 300, 299), (2, 20000, 9), (2, 20000, 19999)):
        q, k, v = _level_case(nq, torch.full((nk,), -float("inf")), 73)
        v[odd, 0, 11] = float("nan")
        for causal in (False, True):
            out, lse, ws = smla.prompt_fwd(q, k, v.cuda(), pc.cu([nq], "cuda"), pc.cu([nk], "cuda"), 1.0, causal=causal)
            assert smla.read_status(ws)[0] == 0 and (out == 0).all() and lse.isneginf().all()
        po, pl = torch.randn(nq, 1, 128, device="cuda"), torch.zeros(nq, 1, device="cuda")
        out, lse, ws = smla.prompt_fwd(q, k, v.cuda(), pc.cu([nq], "cuda"), pc.cu([nk], "cuda"), 1.0, causal=False, prev_out=po, prev_lse=pl,
                                       out_dtype=torch.float32)
        assert torch.equal(out, po) and torch.equal(lse, pl)


# ---------------------------------------------------------------------------- bad bounds
def _guarded(total_q, total_k, n, heads, kv_heads):
    need = smla.prompt_workspace_bytes(total_q, total_k, n, heads, kv_heads)
    raw = torch.full((need + 8192,), 171, dtype=torch.uint8, device="cuda")
    return raw, raw[4096:4096 + need]


def _check_bad(cq, ck, total_q, total_k, heads=2, repeated=False, seed=80):
    """Valid requests keep their results, nothing else is written, neither outputs nor memory around the workspace."""
    q, k, v, pe, _, _ = (t.cuda() for t in pc.prompt_case([total_q], [total_k], heads, heads, 192, True, seed=seed))
    raw, ws = _guarded(total_q, total_k, len(cq) - 1, heads, heads)
    out, lse = torch.full((total_q, heads, 128), 7.0, device="cuda"), torch.full((total_q, heads), 7.0, device="cuda")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    smla.prompt_fwd(q, k, v, i(cq), i(ck), 0.07, k_pe=pe, out=out, lse=lse, ws=ws)
    assert smla.read_status(ws)[0] == 5
    assert (raw[:4096] == 171).all() and (raw[-4096:] == 171).all()
    written, done = torch.zeros(total_q, dtype=torch.bool), set()
    for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
        if not (0 <= a <= b <= total_q and 0 <= c <= d <= total_k) or a == b:
            continue
        written[a:b] = True
        if (a, b, c, d) in done:
            continue
        done.add((a, b, c, d))
        ref = pc.prompt_reference(q[a:b], k[c:d], v[c:d], pe[c:d], pc.cu([b - a]), pc.cu([d - c]), 0.07, True)
        pt.check_rows(out[a:b], lse[a:b], ref)
    assert (out[~written] == 7).all() and (lse[~written] == 7).all()
    ok = smla.prompt_fwd(q, k, v, i([0, total_q]), i([0, total_k]), 0.07, k_pe=pe, ws=ws)  # the workspace is as good as new
    assert smla.read_status(ws)[0] == 0
    ref = pc.prompt_reference(q, k, v, pe, pc.cu([total_q]), pc.cu([total_k]), 0.07, True)
    pt.check_rows(ok[0], ok[1], ref)


@pytest.mark.parametrize("bad", ["backwards", "negative", "past q", "past k", "keys backwards", "none"])
@pytest.mark.parametrize("n,q_len,k_len", [(12, 9, 40), (10, 30, 1100), (3, 2, 9000), (1030, 2, 3)])
def test_prompt_bad_bounds_in_a_plan(bad, n, q_len, k_len):
    """More than eight requests, more than 1,024 keys (cut evenly or not), more requests than the plan's threads."""
    cq, ck = [q_len * i for i in range(n + 1)], [k_len * i for i in range(n + 1)]
    tq, tk = cq[-1], ck[-1]
    if bad == "backwards":
        cq[n // 2] = cq[n // 2 - 1] - 1 if n > 3 else -1
    elif bad == "negative":
        cq[0], ck[0] = -5, -1
    elif bad == "past q":
        cq[n] = tq + 1
    elif bad == "past k":
        ck[n] = tk + 1
    elif bad == "keys backwards":
        ck[1] = ck[2] + 1
    else:
        cq = [-1 - i for i in range(n + 1)]
    # (a bound that is moved lengthens a neighbour or makes requests claim the same rows: those are left out by their bounds)
    if bad == "backwards" and n > 3:
        cq[n // 2] = tq + 5  # past the end for one request, backwards for the next
    _check_bad(cq, ck, tq, tk)


@pytest.mark.parametrize("total_q,total_k,n", [(1500, 700, 9), (1500, 2000, 25), (1100, 9000, 25), (1100, 2000, 1400)])
def test_prompt_bounds_that_overlap_make_more_blocks_than_there_is_room_for(total_q, total_k, n):
    """0 .. total again and again, every other request backwards."""
    cq, ck = [total_q * (i % 2) for i in range(n + 1)], [total_k * (i % 2) for i in range(n + 1)]
    _check_bad(cq, ck, total_q, total_k)


# ---------------------------------------------------------------------------- cache rows
class _Cache:
    def __init__(self, pages, keys=True, seed=90):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.kv_scale, self.kv_dtype = torch.randn(pages, 64, 576, generator=g).to(torch.bfloat16).cuda(), None, "bf16"
        self.k_idx = torch.randn(pages, 64, 64, generator=g).to(torch.bfloat16).cuda() if keys else None
        self.k_idx_scale, self.idx_dtype = None, "bf16" if keys else None


def test_cache_read_status_of_a_small_call_behind_a_large_one():
    """A large call clears the status in a launch of its own, a small one writes it: one after the other in one workspace."""
    c = _Cache(40)
    big, small = torch.arange(40, dtype=torch.int32, device="cuda")[None], torch.full((1, 1), 77, dtype=torch.int32, device="cuda")
    cu_big, cu_small, ws = pc.cu([2560], "cuda"), pc.cu([3], "cuda"), smla.workspace(256)
    lat, pe = (torch.empty(2560, w, dtype=torch.bfloat16, device="cuda") for w in (512, 64))
    for _ in range(200):
        smla.cache_read(c, big, cu_big, 2560, latent=lat, pe=pe, ws=ws)
        smla.cache_read(c, small, cu_small, 3, latent=lat[:3], pe=pe[:3], ws=ws)
        assert smla.read_status(ws)[0] == 5
        smla.cache_read(c, big, cu_big, 2560, latent=lat, pe=pe, ws=ws)
        assert smla.read_status(ws)[0] == 0
    assert torch.equal(lat, c.kv.flatten(0, 1)[:, :512])


def test_calls_on_a_cache_without_indexer_keys():
    """A dense layer's cache: rows appended, read back, attended over in both forms."""
    c = _Cache(6, keys=False)
    tab, lens = torch.tensor([[3, 1], [5, 0]], dtype=torch.int32, device="cuda"), torch.tensor([70, 64], dtype=torch.int32, device="cuda")
    t = [torch.arange(int(n), device="cuda") for n in lens]
    slots = torch.cat([tab[b, i // 64] * 64 + i % 64 for b, i in enumerate(t)]).to(torch.int32)
    pos, table = torch.cat(t).to(torch.int32), smla.rope_table(100)
    rows = (torch.randn(134, 576, generator=torch.Generator().manual_seed(91)) * 2).to(torch.bfloat16).cuda()
    ws = smla.cache_append(c, slots, pos, table, ckv=rows)
    assert smla.read_status(ws)[0] == 0
    lat, pe, keys, ws = smla.cache_read(c, tab, pc.cu([70, 64], "cuda"), 134)
    assert smla.read_status(ws)[0] == 0 and keys is None
    assert torch.equal(lat, rows[:, :512])
    turned, mag = pc.rotate(rows[:, 512:].double().cpu(), table.cpu()[pos.cpu().long()], True)
    pc.check_rotated(pe.cpu(), turned, mag)
    q = torch.randn(2, 64, 576, generator=torch.Generator().manual_seed(92)).to(torch.bfloat16).cuda()
    out, _, ws = smla.shared_prefix_fwd(c, tab, lens, 128, 0, 1, q, 0.04)
    assert smla.read_status(ws)[0] == 0
    for b, (lo, hi) in enumerate(((0, 70), (70, 134))):
        z = (q[b].double() @ torch.cat([lat, pe], 1)[lo:hi].double().T) * 0.04
        ref = torch.softmax(z, 1) @ lat[lo:hi].double()
        assert ((out[b].double() - ref).norm(dim=-1) <= 2.0 ** -7 * ref.norm(dim=-1)).all()
    for call in (lambda: smla.cache_read(c, tab, pc.cu([70, 64], "cuda"), 134, want_keys=True),
                 lambda: smla.cache_append(c, slots, pos, table, ckv=rows, k_idx=rows[:, :64])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(smla.SmlaError):
        smla.indexer_topk(c, tab, lens, 128, 1, rows[:2, None, :64].expand(2, 32, 64).contiguous(), torch.ones(2, 32, device="cuda"), 64)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("idx_dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("n,length", [(3, 70), (9, 333)])
def test_cache_read_of_some_outputs(kv_dtype, idx_dtype, n, length):
    """Every choice of outputs, in small calls and large: the bits of the call for all of them; bad tokens reported alike."""
    width = -(-length // 64)
    c = _filled(n * width, kv_dtype, idx_dtype, 93).to("cuda")
    tab = torch.randperm(n * width, generator=torch.Generator().manual_seed(94)).to(torch.int32).view(n, width).cuda()
    cu, rows = pc.cu([length] * n, "cuda"), n * length
    bad = tab.clone()
    bad[n // 2, 0] = n * width
    for pages, code in ((tab, 0), (bad, 5)):
        *whole, ws = smla.cache_read(c, pages, cu, rows, want_keys=True)
        assert smla.read_status(ws)[0] == code
        for some in range(1, 8):
            a, b, k = bool(some & 1), bool(some & 2), bool(some & 4)
            *got, ws = smla.cache_read(c, pages, cu, rows, want_latent=a, want_pe=b, want_keys=k)
            assert smla.read_status(ws)[0] == code
            for g, w, want in zip(got, whole, (a, b, k)):
                assert torch.equal(g, w) if want else g is None
    x, k = _bf16_rows(c.to("cpu"))
    at = torch.cat([tab[b, torch.arange(length) // 64].cpu().long() * 64 + torch.arange(length) % 64 for b in range(n)])
    good = smla.cache_read(c, tab, cu, rows, want_keys=True)
    assert torch.equal(good[0].cpu(), x[at, :512]) and torch.equal(good[1].cpu(), x[at, 512:]) and torch.equal(good[2].cpu(), k[at])
    with pytest.raises(smla.SmlaError):
        smla.cache_read(c, tab, cu, rows, want_latent=False, want_pe=False)


@pytest.mark.parametrize("ql,kl", [([70, 9], [90, 20]), ([300], [900]), ([2, 1], [9000, 300]), ([200], [20000])])
@pytest.mark.parametrize("join", [False, True])
def test_prompt_without_lse(ql, kl, join):
    q, k, v, pe, cq, ck = (t.cuda() for t in pc.prompt_case(ql, kl, 4, 4, 192, True, seed=95))
    prev = dict(prev_out=torch.randn(sum(ql), 4, 128, device="cuda"), prev_lse=torch.randn(sum(ql), 4, device="cuda") + 5) if join else {}
    out, lse, _ = smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, **prev)
    got, none, ws = smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, want_lse=False, **prev)
    assert smla.read_status(ws)[0] == 0 and none is None and torch.equal(got, out)


def test_calls_without_rows_or_keys_are_refused():
    """As the header says: there is nothing to launch."""
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    c, tab = _Cache(2), i(0, 1)[None]
    for call in (lambda: smla.prompt_fwd(b(0, 2, 192), b(5, 2, 192), b(5, 2, 128), i(0, 0), i(0, 5), 0.1),
                 lambda: smla.prompt_fwd(b(5, 2, 192), b(0, 2, 192), b(0, 2, 128), i(0, 5), i(0, 0), 0.1, causal=False),
                 lambda: smla.prompt_fwd(b(5, 2, 192), b(5, 2, 192), b(5, 2, 128), i(0), i(0), 0.1),
                 lambda: smla.cache_read(c, tab, i(0, 0), 0), lambda: smla.rope_table(0),
                 lambda: smla.rope_apply(b(0, 2, 64), torch.zeros(0, dtype=torch.int32, device="cuda"), smla.rope_table(4))):
        with pytest.raises(smla.SmlaError) as e:
            call()
        assert e.value.code == 1


# ---------------------------------------------------------------------------- another stream
def _stream_calls():
    """Every call that makes tensors of its own, by name: call(stream) -> what it made."""
    g = torch.Generator().manual_seed(96)
    rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    c, tab = _Cache(4), i(0, 1, 2, 3)[None]
    pos, table = torch.arange(200, dtype=torch.int32, device="cuda"), smla.rope_table(256)
    q, k, v, cu, ckv, pe = rn(2, 4, 192), rn(3000, 4, 192), rn(3000, 4, 128), pc.cu([2], "cuda"), rn(200, 576), rn(200, 16, 64)
    ck, qi, w, ql, cu_rows, raw, big = pc.cu([3000], "cuda"), rn(2, 32, 64), torch.ones(2, 32, device="cuda"), rn(2, 64, 576), pc.cu([200], "cuda"), rn(200, 32, 64), rn(200, 4, 64)
    lens, new, free, idx, w200 = i(200), i(3), i(3, 2, 1), torch.zeros(2, 64, dtype=torch.int32, device="cuda"), torch.ones(200, 32, device="cuda")
    return {
        "rope_table": lambda s: [smla.rope_table(256, stream=s)],
        "rope_apply": lambda s: smla.rope_apply(big, pos, table, stream=s),
        "cache_read": lambda s: smla.cache_read(c, tab, cu_rows, 200, want_keys=True, stream=s),
        "prompt_fwd": lambda s: smla.prompt_fwd(q, k, v, cu, ck, 0.07, stream=s),
        "build_tables": lambda s: smla.build_tables(lens, new, tab, free, 8, stream=s),
        "cache_append": lambda s: [smla.cache_append(c, pos, pos, table, ckv=ckv, stream=s)],
        "query_prep": lambda s: smla.query_prep(pos, table, q_pe=pe, q_idx_raw=raw, w=w200, idx_dtype="bf16", stream=s),
        "shared_prefix_fwd": lambda s: smla.shared_prefix_fwd(c, tab, lens, 256, 0, 2, ql, 0.04, stream=s),
        "indexer_topk": lambda s: smla.indexer_topk(c, tab, lens, 256, 2, qi, w, 64, want_scores=True, stream=s),
        "sparse_mla_fwd": lambda s: smla.sparse_mla_fwd(c, tab, ql, idx, 0.04, seq_lens=lens, stream=s),
        "sparse_mla_prefill": lambda s: [t for t in smla.sparse_mla_prefill(c, tab[0], 198, ql, qi, w, 64, 0.04, stream=s) if t is not None],
        "sparse_mla_decode": lambda s: [t for t in smla.sparse_mla_decode(c, tab, lens, 256, 2, ql, qi, w, 64, 0.04, stream=s) if t is not None],
    }


@pytest.mark.parametrize("handle", [False, True])
def test_what_a_call_on_another_stream_makes_outlives_its_work(handle):
    """Outputs and workspaces that the caller drops at once are not handed out again while the stream still works on them.
    (Nothing is written to what is handed out.)"""
    calls = _stream_calls()
    side = torch.cuda.Stream()
    lost = []
    for name, call in calls.items():
        call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # some 100 ms
        made = call(side.cuda_stream if handle else side)
        held = [(t.data_ptr(), t.numel() * t.element_size()) for t in made]
        del made
        fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in held for _ in range(3)]
        assert not side.query(), "the stream was to be busy until here"
        for p, n in held:
            if any(f.data_ptr() < p + n and p < f.data_ptr() + f.numel() for f in fresh):
                lost.append(name)
                break
        torch.cuda.synchronize()
        del fresh
    assert not lost, lost


# ---------------------------------------------------------------------------- rotation tables
@pytest.mark.parametrize("magnitude", [1.0, -1.0, 1.37])
@pytest.mark.parametrize("n,dim,first,kw", [(4099, 64, 0, {}), (70, 256, 1000003, {}), (1001, 8, 1 << 26, dict(base=500.0)),
                                            (2048, 128, 5, dict(base=1e6, factor=8.0, original=8192))])
def test_rope_table_bound(n, dim, first, kw, magnitude):
    """The series' bound. The angle, within an eighth of a turn after exact steps, is a float: its integer, the constant
    2 pi and their product are rounded, 2.5 half steps of 2^-24 relative at most; times an eighth of a turn (0.79) and the slope there
    (0.71) that is 1.4 * 2^-24. The polynomials' last steps are off by 2^-25 each, two for the sine, which is at most 0.71 there, and the
    inner ones by less than 2^-26 together: 2.4 * 2^-24; what the series leaves out is 2^-29. 3 * 2^-24, and a magnitude that is no power of two rounds
    once more. The frequencies (64-bit roundings here and in the reference): 2^-51 of an angle of first + n radians at most."""
    got = smla.rope_table(n, dim, first=first, magnitude=magnitude, **kw).double().cpu()
    ref = pc.table_reference(n, dim, first, magnitude=magnitude, **kw)
    far = (first + n) * 2.0 ** -51
    steps = 3 if abs(magnitude) == 1 else 4
    assert ((got - ref).abs() <= (steps * pc.FP32 + far) * abs(magnitude)).all()


# ---------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("heads,kv_heads", [(128, 1), (1024, 8), (384, 1), (96, 1), (7, 7), (1000, 8), (5, 1)])
@pytest.mark.parametrize("ql,kl", [([1, 6], [1, 300]), ([9], [2000])])
def test_prompt_head_groups(heads, kv_heads, ql, kl):
    """Groups of 128 heads in a tile and more, groups that no power of two fills."""
    c = [t.cuda() for t in pc.prompt_case(ql, kl, heads, kv_heads, 128, True, seed=97)]
    q, k, v, pe, cq, ck = c
    out, lse, ws = smla.prompt_fwd(q, k, v, cq, ck, 0.09, k_pe=pe)
    assert smla.read_status(ws)[0] == 0
    ref = pc.prompt_reference(*c, 0.09, True)
    pc.check_prompt(out, lse, ref)
    pt.check_rows(out, lse, ref)


def test_prompt_offsets_that_pass_32_bits():
    """Queries and results of 2.6e9 values, keys and values of 3.3e9: the first request and the last ones."""
    n, heads = 5000, 1024
    g = torch.Generator(device="cuda").manual_seed(98)
    q = torch.zeros(4 * n, heads, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(40 * n, 64, 256, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, 4), slice(4 * n - 8, 4 * n)]
    for r in ends:
        q[r] = torch.randn(q[r].shape, generator=g, device="cuda").to(torch.bfloat16)
    keys = [slice(0, 40), slice(40 * n - 80, 40 * n)]
    for r in keys:
        kv[r] = torch.randn(kv[r].shape, generator=g, device="cuda").to(torch.bfloat16)
    assert q.numel() > 2 ** 31 and kv.numel() > 2 ** 31
    cq, ck = (torch.arange(0, (n + 1) * m, m, dtype=torch.int32, device="cuda") for m in (4, 40))
    out, lse, ws = smla.prompt_fwd(q, kv[..., :128], kv[..., 128:], cq, ck, 0.09)
    assert smla.read_status(ws)[0] == 0
    for r, s, m in zip(ends, keys, (1, 2)):
        ref = pc.prompt_reference(q[r], kv[s][..., :128], kv[s][..., 128:], None, pc.cu([4] * m), pc.cu([40] * m), 0.09, True)
        pt.check_rows(out[r], lse[r], ref)
    assert (out[4:4 * n - 8] == 0).all()


def test_row_calls_with_offsets_that_pass_32_bits():
    g = torch.Generator(device="cuda").manual_seed(99)
    rows = 180000
    x = torch.zeros(rows, 64, 192, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    for r in (slice(0, 5), slice(rows - 5, rows)):
        x[r] = torch.randn(5, 64, 192, generator=g, device="cuda").to(torch.bfloat16)
    was = {i: x[i].clone() for i in (0, rows - 1)}
    pos, table = torch.full((rows,), 77, dtype=torch.int32, device="cuda"), smla.rope_table(100)
    _, ws = smla.rope_apply(x[..., 128:], pos, table, out=x[..., 128:])
    assert smla.read_status(ws)[0] == 0
    for i, w in was.items():
        ref, mag = pc.rotate(w[:, 128:].double().cpu(), table[77].cpu()[None], True)
        pc.check_rotated(x[i][:, 128:].cpu(), ref, mag)
        assert torch.equal(x[i][:, :128], w[:, :128])
    del x
    pages = 70000
    c = _Cache(1)
    c.kv = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    assert c.kv.numel() > 2 ** 31
    c.k_idx = None
    c.kv[pages - 1] = torch.randn(64, 576, generator=g, device="cuda").to(torch.bfloat16)
    tab = torch.full((1, 3), pages - 1, dtype=torch.int32, device="cuda")
    lat, pe, _, ws = smla.cache_read(c, tab, pc.cu([100], "cuda"), 100, starts=torch.tensor([64], dtype=torch.int32, device="cuda"))
    assert smla.read_status(ws)[0] == 0
    assert torch.equal(torch.cat([lat, pe], 1), c.kv[pages - 1].repeat(2, 1)[:100])


# ---------------------------------------------------------------------------- graphs and threads
@pytest.mark.parametrize("before,after,total_q,total_k", [
    (([70, 9], [90, 20]), ([3, 60], [5, 200]), 100, 220),              # without a plan
    (([300, 40, 0], [900, 60, 0]), ([1, 200, 500], [1, 800, 500]), 800, 1400),
    (([2, 1, 5], [9000, 3, 17000]), ([5, 0, 1], [40, 0, 25000]), 8, 26100)])  # cut elsewhere
def test_prompt_graph_replayed_on_other_bounds(before, after, total_q, total_k):
    """The work is planned on the GPU: a captured call takes the bounds that it finds, bad ones too."""
    q, k, v, pe, _, _ = (t.cuda() for t in pc.prompt_case([total_q], [total_k], 4, 4, 192, True, seed=100))
    n = len(before[0])
    cq, ck = pc.cu(before[0], "cuda"), pc.cu(before[1], "cuda")
    out, lse = torch.zeros(total_q, 4, 128, device="cuda"), torch.zeros(total_q, 4, device="cuda")
    ws = smla.workspace(smla.prompt_workspace_bytes(total_q, total_k, n, 4, 4))
    call = lambda: smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, out=out, lse=lse, ws=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for ql, kl in (before, after, before):
        cq.copy_(pc.cu(ql)), ck.copy_(pc.cu(kl))
        out.fill_(7.0), lse.fill_(7.0)
        g.replay()
        assert smla.read_status(ws)[0] == 0
        rows = sum(ql)
        ref = pc.prompt_reference(q[:rows], k, v, pe, cq, ck, 0.07, True)
        pt.check_rows(out[:rows], lse[:rows], ref)
        assert (out[rows:] == 7).all() and (lse[rows:] == 7).all()
        cq[0] = -1
        g.replay()
        assert smla.read_status(ws)[0] == 5


def test_calls_from_several_threads():
    """Each with a stream and a workspace of its own."""
    import threading
    cases = [([200 + 30 * i], [200 + 30 * i]) if i % 2 else ([2, 3], [3000 + 500 * i, 40]) for i in range(6)]
    data = [[t.cuda() for t in pc.prompt_case(ql, kl, 4, 4, 192, True, seed=101 + i)] for i, (ql, kl) in enumerate(cases)]
    alone = [smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe)[:2] for q, k, v, pe, cq, ck in data]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        q, k, v, pe, cq, ck = data[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                out, lse, ws = smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe)
                if smla.read_status(ws)[0] or not torch.equal(out, alone[i][0]) or not torch.equal(lse, alone[i][1]):
                    bad.append(i)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
