"""The expanded-prompt operators on the GPU against 64-bit references (prompt_common)."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
import prompt_common as pc
import serve_common as sc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    smla.build()


def _cu(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------------------- rotation tables
@pytest.mark.parametrize("n,dim,first,kw", [
    (1, 64, 0, {}), (7, 8, 3, {}), (1000, 64, 0, {}), (333, 128, 100, dict(base=1e6)), (65, 256, 7, {}), (129, 96, 0, {}),
    (500, 64, 1048576, dict(factor=4.0)), (3001, 64, 2000000, dict(factor=32.0, original=32768, magnitude=1.35)),
    (77, 32, 0, dict(factor=2.5, original=4096, beta_fast=16.0, beta_slow=2.0)), (9, 64, 0, dict(magnitude=0.0)),
    (40, 64, 0, dict(factor=3.0, original=6))])  # (every pair on one side of the ramp)
def test_rope_table(n, dim, first, kw):
    raw = torch.full((n * dim + 64,), 5.0, device="cuda")
    got = smla.rope_table(n, dim, first=first, out=raw[32:-32].view(n, dim), **kw)
    ref = pc.table_reference(n, dim, first, **kw)
    # sincospif within a step (2^-24 below 1) and two more roundings of half a step; the angle to 2^-30
    assert ((got.double().cpu() - ref).abs() <= 2.0 ** -22 * abs(kw.get("magnitude", 1.0))).all()
    assert (raw[:32] == 5).all() and (raw[-32:] == 5).all()


def test_rope_table_is_what_the_cache_calls_take():
    """The same rotation as a table made in torch, to a rounding: query_prep on either."""
    t, pos = smla.rope_table(1000), torch.tensor([0, 1, 999], dtype=torch.int32, device="cuda")
    assert (t.cpu() - sc.rope_table(1000)).abs().max() <= 2.0 ** -22
    pe = torch.randn(3, 16, 64, device="cuda").to(torch.bfloat16)
    a, _, _, _ = smla.query_prep(pos, t, q_pe=pe)
    b, _ = smla.rope_apply(pe, pos, t)
    assert torch.equal(a[..., 512:], b)


# ---------------------------------------------------------------------------- rotation
@pytest.mark.parametrize("rows,heads,dim,width,at,inter", [
    (1, 1, 64, 64, 0, True), (1, 5, 8, 16, 8, False), (3, 64, 64, 192, 128, True), (130, 16, 128, 128, 0, False), (33, 7, 96, 104, 8, True),
    (5, 3, 256, 256, 0, False), (515, 2, 32, 192, 64, False), (4500, 4, 64, 64, 0, True)])
@pytest.mark.parametrize("place", ["new", "in place", "strided"])
def test_rope_apply(rows, heads, dim, width, at, inter, place):
    g = torch.Generator().manual_seed(rows + dim)
    wide = (torch.randn(rows, heads, width, generator=g) * 3).to(torch.bfloat16)
    pos = torch.randint(0, 700, (rows,), generator=g, dtype=torch.int32)
    pos[rows // 2] = -1
    tab = smla.rope_table(700, dim)
    x = wide.cuda()
    part = x[..., at:at + dim]
    if place == "in place":
        out = part
    elif place == "strided":
        out = torch.full((rows, heads, dim + 24), 9.0, dtype=torch.bfloat16, device="cuda")[..., 8:8 + dim]
    else:
        out = torch.full((rows, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    got, ws = smla.rope_apply(part, pos.cuda(), tab, interleaved=inter, out=out)
    assert smla.read_status(ws)[0] == 0
    live = torch.arange(rows) != rows // 2
    src = wide[..., at:at + dim].double()
    ref, mag = pc.rotate(src, tab.cpu()[pos.clamp_min(0).long()][:, None], inter)
    pc.check_rotated(got.cpu()[live], ref[live], mag[live])
    skipped = got[rows // 2].double().cpu()
    assert torch.equal(skipped, src[rows // 2]) if place == "in place" else (skipped == 9).all()
    if place == "in place":  # the rest of the heads
        rest = torch.ones(width, dtype=torch.bool)
        rest[at:at + dim] = False
        assert torch.equal(x.cpu()[..., rest], wide[..., rest])
    elif place == "strided":
        whole = out._base
        assert (whole[..., :8] == 9).all() and (whole[..., 8 + dim:] == 9).all()


@pytest.mark.parametrize("rows", [4, 5000])
def test_rope_apply_reports_positions(rows):
    tab, x = smla.rope_table(10, 64), torch.ones(rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pos[1], pos[2], pos[3] = 10, -1, -7
    out, ws = smla.rope_apply(x, pos, tab, out=torch.full_like(x, 7.0))
    assert smla.read_status(ws)[0] == 5
    assert (out[1:4] == 7).all() and (out[0] == 1).all() and (out[4:] == 1).all()
    out, ws = smla.rope_apply(x[:1], pos[:1], tab, ws=ws)
    assert smla.read_status(ws)[0] == 0


# ---------------------------------------------------------------------------- cache rows
def _filled(pages, kv_dtype, idx_dtype, seed, key_scale=True):
    c = sc.filled_cache(pages, kv_dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    if idx_dtype == "fp8":
        c.k_idx = torch.randn(pages, 64, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
        c.k_idx_scale = torch.rand(pages, 64, generator=g) + 0.1 if key_scale else None
    else:
        c.k_idx, c.k_idx_scale = torch.randn(pages, 64, 64, generator=g).to(torch.bfloat16), None
    c.idx_dtype = idx_dtype
    return c


def _bf16_rows(c):
    """What the cache's rows are as bf16: codes times scales in fp32, rounded once. [pool rows, ..]"""
    f8 = lambda t: t.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    kv = c.kv.flatten(0, 1)
    if c.kv_dtype == "bf16":
        x = kv
    elif c.kv_dtype == "fp8":
        x = (f8(kv) * c.kv_scale.flatten()[:, None]).to(torch.bfloat16)
    else:
        s = kv[:, 512:528].contiguous().view(torch.float32).repeat_interleave(128, 1)
        x = torch.cat([(f8(kv[:, :512]) * s).to(torch.bfloat16), kv[:, 528:].contiguous().view(torch.bfloat16)], 1)
    k = c.k_idx.flatten(0, 1)
    if c.idx_dtype == "fp8":
        k = f8(k)
        k = (k if c.k_idx_scale is None else k * c.k_idx_scale.flatten()[:, None]).to(torch.bfloat16)
    return x, k


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
@pytest.mark.parametrize("lens,starts,idx_dtype", [([1], [0], "fp8"), ([64], [63], "bf16"), ([0, 33, 0, 1, 0], [5, 40, 0, 127, 9], "fp8"),
                                                   ([200, 31, 32, 65], [0, 1, 64, 130], "bf16"), ([3] * 70 + [0] * 5, list(range(75)), "fp8")])
def test_cache_read(kv_dtype, lens, starts, idx_dtype):
    n, width = len(lens), max(-(-(a + b) // 64) for a, b in zip(lens, starts)) + 1
    pages = sum(-(-(a + b) // 64) for a, b in zip(lens, starts)) + 2
    c = _filled(pages, kv_dtype, idx_dtype, n, key_scale=n != 5)
    perm, at = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32), 0
    tab = torch.full((n, width), -1, dtype=torch.int32)
    rows = []
    for b in range(n):
        k = -(-(lens[b] + starts[b]) // 64)
        tab[b, :k] = perm[at:at + k]
        at += k
        t = torch.arange(starts[b], starts[b] + lens[b])
        rows.append(tab[b, t // 64].long() * 64 + t % 64)
    rows, cu = torch.cat(rows), pc.cu(lens)
    d, total = c.k_idx.shape[-1], sum(lens)
    new = lambda w, pad: torch.full((total + 9, w + pad), 7.0, dtype=torch.bfloat16, device="cuda")[:, :w]  # noqa: E731
    lat, pe, keys = new(512, 8), new(64, 0), new(d, 64)
    cg = c.to("cuda")
    *_, ws = smla.cache_read(cg, tab.cuda(), cu.cuda(), total + 9, starts=torch.tensor(starts, dtype=torch.int32).cuda(), latent=lat, pe=pe, keys=keys)
    assert smla.read_status(ws)[0] == 0
    x, k = _bf16_rows(c)
    for got, ref in ((lat, x[rows, :512]), (pe, x[rows, 512:]), (keys, k[rows])):
        assert torch.equal(got[:total].cpu(), ref)
        assert (got[total:] == 7).all() and (got._base[:, got.shape[1]:] == 7).all()
    if all(s == 0 for s in starts) or n == 4:  # without a list of starts
        lat2, pe2, none, _ = smla.cache_read(cg, tab.cuda(), cu.cuda(), total)
        base = torch.cat([tab[b, torch.arange(lens[b]) // 64].long() * 64 + torch.arange(lens[b]) % 64 for b in range(n)])
        assert none is None and torch.equal(lat2.cpu(), x[base, :512]) and torch.equal(pe2.cpu(), x[base, 512:])


def test_cache_read_reports_what_is_not_there():
    c = _filled(4, "fp8", "fp8", 5).to("cuda")
    tab = torch.tensor([[0, 9], [1, -1], [2, 3]], dtype=torch.int32).cuda()
    starts = torch.tensor([60, 0, 126], dtype=torch.int32).cuda()
    def read(cu, rows, st=starts):
        out = [torch.full((rows, w), 7.0, dtype=torch.bfloat16, device="cuda") for w in (512, 64)]
        *_, ws = smla.cache_read(c, tab, torch.tensor(cu, dtype=torch.int32).cuda(), rows, starts=st, latent=out[0], pe=out[1])
        return out[0].float().cpu(), smla.read_status(ws)[0]
    x, _ = _bf16_rows(c.to("cpu"))
    got, rc = read([0, 8, 10, 13], 13)  # page 9 is no page; request 2 ends past its table
    assert rc == 5
    assert torch.equal(got[:4], x[60:64, :512].float()) and (got[4:8] == 0).all()
    assert torch.equal(got[8:10], x[64:66, :512].float())
    assert torch.equal(got[10:12], x[3 * 64 + 62:4 * 64, :512].float()) and (got[12] == 0).all()
    got, rc = read([0, 4, 6, 9], 7)  # more rows than there is room for
    assert rc == 5 and (got[:6] != 7).any(1).all() and torch.equal(got[6], x[3 * 64 + 62, :512].float())
    got, rc = read([2, 4, 3, 5], 8)  # runs backwards; rows before the first and behind the last are left
    assert rc == 5 and (got[:2] == 7).all() and (got[5:] == 7).all()
    got, rc = read([-3, 0, 2, 3], 4)
    assert rc == 5 and (got[3] == 7).all()
    got, rc = read([0, 0, 0, 0], 2)
    assert rc == 0 and (got == 7).all()
    got, rc = read([0, 2, 2, 2], 2, torch.tensor([-1, 0, 0], dtype=torch.int32).cuda())
    assert rc == 5 and (got[0] == 0).all() and torch.equal(got[1], x[0, :512].float())


@pytest.mark.parametrize("n,length", [(1, 1000), (1, 1100), (1200, 1), (40, 25), (41, 25)])
def test_cache_read_reports_the_same_in_small_and_large_calls(n, length):
    """One missing page anywhere among the rows; a list that ends past the outputs."""
    c = _filled(30, "bf16", "fp8", 41).to("cuda")
    width = -(-length // 64)
    tables = lambda: (torch.arange(n * width, dtype=torch.int32) % 30).view(n, width)  # noqa: E731
    cu = pc.cu([length] * n)
    for at in (0, n * width // 2, n * width - 1):
        tab = tables()
        tab.view(-1)[at] = 30
        lat, _, _, ws = smla.cache_read(c, tab.cuda(), cu.cuda(), n * length)
        assert smla.read_status(ws)[0] == 5
        b, p = at // width, at % width
        gone = slice(b * length + 64 * p, b * length + min(length, 64 * (p + 1)))
        assert (lat[gone] == 0).all() and (lat != 0).any(1).sum() == n * length - (gone.stop - gone.start)
    lat, _, _, ws = smla.cache_read(c, tables().cuda(), cu.cuda(), n * length, ws=ws)
    assert smla.read_status(ws)[0] == 0 and (lat != 0).any(1).all()
    cu[n] += 1
    _, _, _, ws = smla.cache_read(c, tables().cuda(), cu.cuda(), n * length, ws=ws)
    assert smla.read_status(ws)[0] == 5


def test_row_calls_on_a_stream_and_in_a_graph():
    """Captured, replayed on changed inputs and on a side stream: what a plain call gives; the status of a bad replay, and
    of a good one after it."""
    c = _filled(6, "fp8", "fp8", 40).to("cuda")
    tab = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32).cuda()
    cu, starts = pc.cu([70, 30], "cuda"), torch.tensor([0, 64], dtype=torch.int32).cuda()
    pos, table = torch.arange(100, dtype=torch.int32, device="cuda"), torch.empty(200, 64, device="cuda")
    lat, pe, out = (torch.zeros(100, *w, dtype=torch.bfloat16, device="cuda") for w in ((512,), (64,), (1, 64)))
    ws = [smla.workspace(256) for _ in range(2)]

    def call():
        smla.rope_table(200, out=table)
        smla.cache_read(c, tab, cu, 100, starts=starts, latent=lat, pe=pe, ws=ws[0])
        smla.rope_apply(pe[:, None], pos, table, out=out, ws=ws[1])

    def expect():
        x, _ = _bf16_rows(c.to("cpu"))
        b, t = (torch.arange(100) >= 70).long(), torch.cat([torch.arange(70), torch.arange(30)]) + starts.cpu().repeat_interleave(torch.tensor([70, 30]))
        rows = x[tab.cpu()[b, t // 64].long() * 64 + t % 64]
        assert torch.equal(lat.cpu(), rows[:, :512]) and torch.equal(pe.cpu(), rows[:, 512:])
        ref, mag = pc.rotate(rows[:, 512:].double(), table.cpu()[pos.cpu().long()], True)
        pc.check_rotated(out.cpu()[:, 0], ref, mag)

    call()
    expect()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    tab.copy_(tab.flip(0).clone())
    starts.copy_(torch.tensor([100, 3], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            g.replay()
    side.synchronize()
    expect()
    assert smla.read_status(ws[0])[0] == 0 and smla.read_status(ws[1])[0] == 0
    held = int(tab[1, 0])
    tab[1, 0] = 77
    pos[5] = 200
    g.replay()
    assert smla.read_status(ws[0])[0] == 5 and smla.read_status(ws[1])[0] == 5
    tab[1, 0] = held
    pos[5] = 5
    g.replay()
    torch.cuda.synchronize()
    expect()
    assert smla.read_status(ws[0])[0] == 0 and smla.read_status(ws[1])[0] == 0


# ---------------------------------------------------------------------------- attention
def _run(q, k, v, pe, cq, ck, scale, causal, status=0, **kw):
    kv = k._base.cuda() if k._base is not None else None  # keys and values side by side, as they are here
    dk = k.shape[-1]
    k, v = (kv[..., :dk], kv[..., dk:]) if kv is not None else (k.cuda(), v.cuda())
    out, lse, ws = smla.prompt_fwd(q.cuda(), k, v, cq.cuda(), ck.cuda(), scale, k_pe=_cu(pe), causal=causal, **kw)
    assert smla.read_status(ws)[0] == status
    return out, lse


FORMS = [(192, True), (192, False), (128, False), (128, True)]


@pytest.mark.parametrize("d,pe", FORMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,heads,kv_heads", [
    ([1], [1], 1, 1), ([1], [300], 2, 2), ([128], [128], 2, 1), ([129], [129], 2, 2), ([255, 1], [256, 2], 2, 2), ([257], [400], 3, 1),
    ([0, 5, 0, 130, 1], [0, 5, 7, 131, 400], 4, 2),      # empty requests
    ([10, 3], [4, 0], 4, 4),                             # tokens that see nothing
    ([33], [700], 16, 1), ([7, 90], [300, 90], 12, 4), ([64, 64, 64], [64, 128, 192], 8, 8)])
def test_prompt(d, pe, causal, ql, kl, heads, kv_heads):
    c = pc.prompt_case(ql, kl, heads, kv_heads, d, pe, seed=sum(ql) + heads)
    out, lse = _run(*c, d ** -0.5, causal)
    rows = slice(0, sum(ql))
    pc.check_prompt(out, lse, pc.prompt_reference(*c, d ** -0.5, causal), rows)


@pytest.mark.parametrize("heads,kv_heads,n,length", [(64, 64, 1, 1500), (64, 8, 3, 1100), (16, 16, 2, 2500), (64, 1, 1, 700)])
def test_prompt_long(heads, kv_heads, n, length):
    ql = [length - 37 * i for i in range(n)]
    q, k, v, pe, cq, ck = pc.prompt_case(ql, ql, heads, kv_heads, 192, True, seed=heads)
    out, lse = _run(q, k, v, pe, cq, ck, 192 ** -0.5, True)
    ref = pc.prompt_reference(*(t.cuda() for t in (q, k, v, pe, cq, ck)), 192 ** -0.5, True)
    pc.check_prompt(out, lse, ref)


@pytest.mark.parametrize("ql,kl,heads,kv_heads,causal", [([1], [40000], 1, 1, True), ([1, 2], [20011, 9000], 64, 64, True), ([5], [30000], 16, 1, False),
                                                         ([300], [20000], 4, 4, True), ([1] * 9, [5000 + 777 * i for i in range(9)], 8, 2, False)])
def test_prompt_few_rows_many_keys(ql, kl, heads, kv_heads, causal):
    """Keys that are cut into pieces."""
    q, k, v, pe, cq, ck = pc.prompt_case(ql, kl, heads, kv_heads, 192, True, seed=heads + sum(ql))
    out, lse = _run(q, k, v, pe, cq, ck, 192 ** -0.5, causal)
    ref = pc.prompt_reference(*(t.cuda() for t in (q, k, v, pe, cq, ck)), 192 ** -0.5, causal)
    pc.check_prompt(out, lse, ref)


def test_prompt_strides_and_padding():
    """Queries inside wider rows, rows behind the last request (left as they are), bounds that begin later."""
    ql, kl = [40, 3], [90, 200]
    q, k, v, pe, _, _ = pc.prompt_case(ql, kl, 8, 8, 192, True, seed=3, extra_q=30, extra_k=50)
    cq, ck = torch.tensor([0, 40, 43], dtype=torch.int32), torch.tensor([0, 90, 290], dtype=torch.int32)
    wide = torch.zeros(q.shape[0], 8, 256, dtype=torch.bfloat16, device="cuda")
    wide[..., 64:] = q.cuda()
    out = torch.full((q.shape[0], 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], 8), 7.0, device="cuda")
    kc, vc = k.cuda(), v.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # values by head
    pew = torch.zeros(pe.shape[0], 576, dtype=torch.bfloat16, device="cuda")
    pew[:, 512:] = pe.cuda()
    _, _, ws = smla.prompt_fwd(wide[..., 64:], kc, vc if vc.stride(0) >= 128 else v.cuda(), cq.cuda(), ck.cuda(), 0.07, k_pe=pew[:, 512:], out=out, lse=lse)
    assert smla.read_status(ws)[0] == 0
    ref = pc.prompt_reference(q, k, v, pe, cq, ck, 0.07, True)
    pc.check_prompt(out, lse, ref, slice(0, 43))
    assert (out[43:] == 7).all() and (lse[43:] == 7).all()
    cq2, ck2 = cq + 5, ck + 7  # rows 0..4 belong to no request
    out.fill_(7.0)
    smla.prompt_fwd(wide[..., 64:], kc, v.cuda(), cq2.cuda(), ck2.cuda(), 0.07, k_pe=pew[:, 512:], out=out, lse=lse)
    assert (out[:5] == 7).all() and (out[48:] == 7).all()
    ref = pc.prompt_reference(q[5:], k[7:], v[7:], pe[7:], cq, ck, 0.07, True)
    pc.check_prompt(out[5:], lse[5:], ref, slice(0, 30))


@pytest.mark.parametrize("bad", ["values", "keys", "inf", "mixed"])
@pytest.mark.parametrize("n,at", [(70, [69]), (300, [299, 150]), (260, [3, 128, 255, 256])])
def test_prompt_what_is_not_finite_stays_with_those_that_see_it(bad, n, at):
    q, k, v, pe, cq, ck = pc.prompt_case([n, 20], [n, 20], 4, 2, 192, True, seed=n)
    for i, j in enumerate(at):
        if bad == "keys":
            k[j, 1, 5] = float("nan")
        elif bad == "values":
            v[j, 0, 3 + i] = float("nan")
        elif bad == "inf":
            v[j, 1, 100] = float("inf") if i % 2 == 0 else float("-inf")
        else:
            v[j, i % 2, 64], pe[j, 9] = float("-inf"), float("inf")
    out, lse = _run(q, k, v, pe, cq, ck, 0.07, True)
    clean = pc.prompt_reference(torch.nan_to_num(q), torch.nan_to_num(k), v, torch.nan_to_num(pe, 0.0, 0.0, 0.0), cq, ck, 0.07, True)
    if bad in ("values", "inf"):
        pc.check_prompt(out, lse, clean)
        return
    sees = torch.zeros(n + 20, dtype=torch.bool)
    sees[min(at):n] = True  # logits that are not finite: such rows may hold anything, the others are as if nothing were there
    pc.check_prompt(out, lse, clean, ~sees)
    assert not torch.isfinite(out[at[0], 2:] if bad == "keys" else out[at[0]]).all()


@pytest.mark.parametrize("fp32", [True, False])
def test_prompt_joined_parts_are_the_whole(fp32):
    """Three parts of the keys one after another, in place, against all keys at once."""
    q, k, v, pe, cq, ck = pc.prompt_case([30], [900], 8, 8, 192, True, seed=9)
    cuts = [0, 500, 740, 870]
    args = lambda a, b: (q, k[a:b], v[a:b], pe[a:b], cq, pc.cu([b - a]))  # noqa: E731
    out = lse = None
    g = lambda t: t.cuda()  # noqa: E731
    for a, b in zip(cuts, cuts[1:]):
        out, lse, ws = smla.prompt_fwd(g(q), g(k)[a:b], g(v)[a:b], g(cq), pc.cu([b - a], "cuda"), 0.07, k_pe=g(pe)[a:b], causal=False,
                                       prev_out=out, prev_lse=lse, out=out, lse=lse, out_dtype=torch.float32)
        assert smla.read_status(ws)[0] == 0
    out, lse, ws = smla.prompt_fwd(g(q), g(k)[870:], g(v)[870:], g(cq), pc.cu([30], "cuda"), 0.07, k_pe=g(pe)[870:], causal=True, prev_out=out,
                                   prev_lse=lse, out=out if fp32 else None, lse=lse)
    ref = pc.prompt_reference(q, k, v, pe, cq, ck, 0.07, True)
    pc.check_prompt(out, lse, ref)


def test_prompt_join_with_nothing():
    """prev_lse of -inf (whatever prev_out holds), rows that see nothing themselves, and both."""
    q, k, v, pe, cq, ck = pc.prompt_case([8], [4], 4, 4, 192, True, seed=10)  # rows 0..3 see no key
    po, pl = torch.randn(8, 4, 128), torch.randn(8, 4)
    pl[::2] = float("-inf")
    po[::2] = float("nan")
    out, lse = _run(q, k, v, pe, cq, ck, 0.07, True, prev_out=po.cuda(), prev_lse=pl.cuda(), out_dtype=torch.float32)
    ref = pc.prompt_reference(q, k, v, pe, cq, ck, 0.07, True, prev=(po, pl))
    pc.check_prompt(out, lse, ref)
    assert torch.allclose(out[1].cpu(), po[1], rtol=2.0 ** -18) and (out[0] == 0).all() and lse[0].isneginf().all()


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1e-6, 0.7])
def test_prompt_softmax_scales(scale):
    c = pc.prompt_case([150, 9], [170, 400], 4, 2, 192, False, seed=11)
    out, lse = _run(*c, scale, True)
    pc.check_prompt(out, lse, pc.prompt_reference(*c, scale, True))


def test_prompt_peaked_and_rising_logits():
    """Logits of up to some hundreds whose running maximum keeps rising."""
    q, k, v, pe, cq, ck = pc.prompt_case([200], [1000], 4, 4, 192, True, seed=12, std=10.0)
    k *= torch.linspace(0.1, 3.0, 1000)[:, None, None].to(torch.bfloat16)
    out, lse = _run(q, k, v, pe, cq, ck, 192 ** -0.5, True)
    pc.check_prompt(out, lse, pc.prompt_reference(q, k, v, pe, cq, ck, 192 ** -0.5, True))


@pytest.mark.parametrize("cq,ck", [([0, 50, 40, 90], [0, 50, 60, 90]), ([0, 30, 60, 101], [0, 30, 60, 90]), ([0, 30, 60, 90], [0, 30, 20, 90]),
                                   ([-4, 30, 60, 90], [0, 30, 60, 90]), ([0, 30, 60, 90], [0, 30, 60, 91])])
def test_prompt_reports_bad_bounds(cq, ck):
    """The requests whose bounds are right keep their results; the others write nothing."""
    q, k, v, pe, _, _ = pc.prompt_case([100], [90], 2, 2, 192, True, seed=13)
    i = lambda a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    out = torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = _run(q, k, v, pe, i(cq), i(ck), 0.07, True, status=5, out=out)
    written = torch.zeros(100, dtype=torch.bool)
    for b in range(3):
        if 0 <= cq[b] <= cq[b + 1] <= 100 and 0 <= ck[b] <= ck[b + 1] <= 90:
            r, s = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
            ref = pc.prompt_reference(q[r], k[s], v[s], pe[s], pc.cu([cq[b + 1] - cq[b]]), pc.cu([ck[b + 1] - ck[b]]), 0.07, True)
            if cq != [0, 50, 40, 90]:  # (there two requests claim the same rows)
                pc.check_prompt(out[r], lse[r], ref)
            written[r] = True
    assert (out.cpu()[~written] == 7).all()


@pytest.mark.parametrize("ql,kl,heads", [([200, 31], [260, 31], 16), ([1], [30000], 16)])
def test_prompt_repeats_on_another_stream_and_in_a_graph(ql, kl, heads):
    """The same bits each time; nothing outside the outputs is written."""
    q, k, v, pe, cq, ck = (t.cuda() for t in pc.prompt_case(ql, kl, heads, heads, 192, True, seed=14))
    tq = sum(ql)
    ws = smla.workspace(smla.prompt_workspace_bytes(tq, sum(kl), len(ql), heads, heads))
    raw = torch.full((tq * heads * 128 + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = raw[2048:-2048].view(tq, heads, 128), torch.empty(tq, heads, device="cuda")
    call = lambda: smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, out=out, lse=lse, ws=ws)  # noqa: E731
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
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, flse)


def test_prompt_two_calls_at_once():
    """Two streams with a workspace each."""
    cases = [[t.cuda() for t in pc.prompt_case([900 + 50 * i], [900 + 50 * i], 16, 16, 192, True, seed=20 + i)] for i in range(2)]
    alone = [smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe)[0] for q, k, v, pe, cq, ck in cases]
    ws = [smla.workspace(smla.prompt_workspace_bytes(1000, 1000, 1, 16, 16)) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(a) for a in alone]
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, k, v, pe, cq, ck), w, s, o in zip(cases, ws, streams, outs):
            with torch.cuda.stream(s):
                smla.prompt_fwd(q, k, v, cq, ck, 0.07, k_pe=pe, out=o, ws=w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs)) and all(smla.read_status(w)[0] == 0 for w in ws)


@pytest.mark.parametrize("d,pe,heads,kv_heads,scale", [(192, True, 4, 4, 0.07), (128, False, 8, 1, 0.09), (192, False, 6, 2, -0.07), (128, True, 2, 2, 0.09)])
def test_prompt_cut_keys_joined_in_place(d, pe, heads, kv_heads, scale):
    """Few rows whose keys are cut into pieces, joined with an earlier result in its own buffers."""
    ql, kl = [2, 1, 5], [9000, 3, 17000]
    c = pc.prompt_case(ql, kl, heads, kv_heads, d, pe, seed=30)
    g = torch.Generator().manual_seed(31)
    po, pl = torch.randn(8, heads, 128, generator=g), torch.randn(8, heads, generator=g) + 8
    pl[4] = float("-inf")
    ref = pc.prompt_reference(*(None if t is None else t.cuda() for t in c), scale, True, prev=(po.cuda(), pl.cuda()))
    out, lse = po.cuda(), pl.cuda()
    _run(*c, scale, True, prev_out=out, prev_lse=lse, out=out, lse=lse)
    pc.check_prompt(out, lse, ref)


@pytest.mark.parametrize("n,length", [(3, 6000), (2, 300), (300, 9000)])
def test_prompt_cut_keys_and_values_that_are_not_finite(n, length):
    """Late values that only some tokens see, where key tiles go to two halves of the pipeline and are cut."""
    q, k, v, pe, cq, ck = pc.prompt_case([n], [length], 2, 1, 192, True, seed=32)
    for i, j in enumerate((length - 1, length - n // 2, length - n)):  # the last token's, some tokens', every token's
        v[j, 0, 5 + 40 * i] = [float("nan"), float("inf"), float("-inf")][i]
    v[length - 1, 0, 45] = float("-inf")  # against the +inf of an earlier key
    out, lse = _run(q, k, v, pe, cq, ck, 0.07, True)
    ref = pc.prompt_reference(*(t.cuda() for t in (q, k, torch.nan_to_num(v, 0.0, 0.0, 0.0), pe, cq, ck)), 0.07, True)
    want = ref[0].clone()
    pos = torch.arange(n, device="cuda") + length - n
    for j in sorted({length - 1, length - n // 2, length - n}):
        bad = ~torch.isfinite(v[j, 0]).cuda()
        sees = pos >= j
        add = torch.where(bad, v[j, 0].cuda().double(), 0.0)
        want[sees] = torch.where(bad, want[sees] + add, want[sees])
    pc.check_prompt(out, lse, (want, *ref[1:]))


def test_prompt_many_requests():
    """More requests than the plan's threads, most of them short, some empty."""
    rng = np.random.default_rng(33)
    ql = rng.integers(0, 4, 2500).tolist()
    kl = (np.array(ql) + rng.integers(0, 5, 2500)).tolist()
    c = pc.prompt_case(ql, kl, 2, 1, 192, True, seed=34)
    out, lse = _run(*c, 0.07, True)
    pc.check_prompt(out, lse, pc.prompt_reference(*c, 0.07, True))


def test_prompt_very_many_keys():
    """More key tiles than the plan's bins."""
    c = pc.prompt_case([2, 70], [140000, 300], 1, 1, 192, True, seed=35)
    out, lse = _run(*c, 0.07, True)
    pc.check_prompt(out, lse, pc.prompt_reference(*(t.cuda() for t in c), 0.07, True))


@pytest.mark.parametrize("fp32", [False, True])
def test_prompt_results_on_a_16_byte_boundary(fp32):
    c = pc.prompt_case([70, 300], [90, 300], 3, 3, 192, True, seed=36)
    t = torch.float32 if fp32 else torch.bfloat16
    pad = 4 if fp32 else 8
    raw = torch.full((370 * 3 * 128 + 64,), 3.0, dtype=t, device="cuda")
    out = raw[pad:pad + 370 * 384].view(370, 3, 128)
    assert out.data_ptr() % 32 == 16
    _, lse = _run(*c, 0.07, True, out=out)
    pc.check_prompt(out, lse, pc.prompt_reference(*c, 0.07, True))
    assert (raw[:pad] == 3).all() and (raw[pad + 370 * 384:] == 3).all()


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
def test_expanded_equals_latent_attention(kv_dtype):
    """The calls as a prompt step uses them: new rows appended to the cache, context and new rows read back, expanded by
    an up-projection, queries rotated, the new tokens' own keys and the context's in two parts joined: against the
    64-bit attention in the latent form over what the cache holds."""
    g = torch.Generator(device="cuda").manual_seed(21)
    heads, ctx, new = 16, [100, 0, 333], [60, 5, 17]
    n, rows = 3, sum(new)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    c = sc.filled_cache(20, kv_dtype, 22).to("cuda")
    c.k_idx_scale.fill_(1.0)
    tab = torch.randperm(20, generator=g, device="cuda")[:18].to(torch.int32).view(3, 6)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = smla.rope_table(1024)
    t0 = tab.clone()
    for b in range(n):
        t0[b, -(-ctx[b] // 64):] = -1
    free = torch.cat([tab[b, -(-ctx[b] // 64):-(-(ctx[b] + new[b]) // 64)] for b in range(n)]).contiguous()
    lens, cu_new, pos, slots, _, _, ws = smla.build_tables(i32(ctx), i32(new), t0, free, rows)
    assert smla.read_status(ws)[0] == 0
    smla.cache_append(c, slots, pos, table, ckv=rn(rows, 576))
    q = rn(rows, heads, 192)
    q0 = q.clone()
    smla.rope_apply(q[..., 128:], pos, table, out=q[..., 128:])
    w = rn(512, heads * 256, std=512 ** -0.5)  # the up-projection: each head's keys and values
    scale, parts = 192 ** -0.5, []
    cu_ctx = pc.cu(ctx, "cuda")
    for cu, starts, causal in ((cu_ctx, None, False), (cu_new, i32(ctx), True)):
        total = int(cu[-1])
        lat, pe, _, ws = smla.cache_read(c, t0, cu, total, starts=starts)
        assert smla.read_status(ws)[0] == 0
        kv = (lat @ w).view(total, heads, 256)
        parts.append((kv[..., :128], kv[..., 128:], pe, cu, causal))
    out = lse = None
    for k, v, pe, cu, causal in parts:
        out, lse, ws = smla.prompt_fwd(q, k, v, cu_new, cu, scale, k_pe=pe, causal=causal, prev_out=out, prev_lse=lse, out_dtype=torch.float32)
        assert smla.read_status(ws)[0] == 0
    # in 64 bits: (q_nope W_k) . latent + q_pe . pe, the weighted latent rows times W_v. The expanded keys and
    # values are rounded to bf16 on the way, the rows too where the cache has 8 bits, and the turned queries: three
    # roundings of 2^-8 / sqrt(3) of a value in the mean square, independent, so logits of about 1 are off by 2^-8 in the
    # mean square and a weighted row by no more than that of its norm: 2^-5 is eight times it.
    kv64 = torch.from_numpy(sc.latent_values(c.to("cpu"))).cuda()
    w64 = w.double().view(512, heads, 256)
    turned, _ = pc.rotate(q0[..., 128:].double().cpu(), table.cpu()[pos.cpu().long()][:, None], True)
    r = 0
    for b in range(n):
        s = torch.arange(ctx[b] + new[b], device="cuda")
        keys = kv64[t0[b, s // 64].long() * 64 + s % 64]
        for i in range(new[b]):
            seen = keys[:ctx[b] + i + 1]
            qa = torch.einsum("hd,lhd->hl", q0[r, :, :128].double(), w64[..., :128])
            z = (qa @ seen[:, :512].T + turned[r].cuda() @ seen[:, 512:].T) * scale
            ref = torch.einsum("hl,lhd->hd", torch.softmax(z, 1) @ seen[:, :512], w64[..., 128:])
            err = (out[r].double() - ref).norm(dim=-1) / ref.norm(dim=-1)
            assert err.max() <= 2.0 ** -5 and (lse[r].double() - torch.logsumexp(z, 1)).abs().max() <= 2.0 ** -5
            r += 1
