"""The serving operators where their contracts end. References: serve_common."""
import numpy as np
import pytest
import torch

import indexer_top_sparse_score_gb300 as smla
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
