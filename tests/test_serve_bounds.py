"""The bounds on whole rows catch a tile of keys that the oracle leaves out (no GPU)."""
import numpy as np
import pytest
import torch

import serve_bounds as sb
import serve_common as sc


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_ds_mla"])
def test_lost_tile_is_caught(kv_dtype):
    n, tile = 38000, np.s_[12800:12928]
    c, tab, sl, q = sc.attention_case(1, 1, 16, kv_dtype, 0, [n], seed=40)
    out, lse, _, _ = sc.attention_reference(c, tab, sl, 1, q, 0, sc.SM_SCALE)
    bf16 = lambda v: torch.from_numpy(v).to(torch.bfloat16).double().numpy()  # noqa: E731
    sb.check_rows(bf16(out), lse, out, lse)
    kv = sc.latent_values(c)[(tab[0].long()[:, None] * 64 + torch.arange(64)).flatten().numpy()[:n]]
    e = np.exp(q[0].float().double().numpy() @ kv.T * sc.SM_SCALE)
    total, part = e.sum(-1, keepdims=True), e[:, tile].sum(-1, keepdims=True)
    values = e[:, tile] @ kv[tile, :512]
    no_product = out[0] - values / total
    no_tile = (out[0] * total - values) / (total - part)
    for h in range(16):  # in any one row
        for lost in (no_product, no_tile):
            a = out.copy()
            a[0, h] = lost[h]
            with pytest.raises(AssertionError, match="values"):
                sb.check_rows(bf16(a), lse, out, lse)
        b = lse.copy()
        b[0, h] = np.log(total - part)[h, 0]
        with pytest.raises(AssertionError, match="lse"):
            sb.check_rows(out, b, out, lse)
