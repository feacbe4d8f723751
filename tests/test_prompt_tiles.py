"""The bounds of prompt_tiles on modelled results (no GPU): right ones pass, ones with a key tile lost or doubled do not."""
import pytest
import torch

import prompt_tiles as pt


def _counted(ql, kl, causal, by, wrong=None):
    """What the kernel would give in fp32, from per-key sums; wrong: (first key, weight) of a tile of the first request."""
    out, lse = [], []
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        w = torch.ones(nk)
        if wrong is not None and b == 0:
            w[wrong[0]:wrong[0] + 128] = wrong[1]
        j = torch.arange(nk)
        v = torch.nn.functional.one_hot((j // 128 if by == "tile" else j) % 128, 128).float()
        upto = torch.cat([torch.zeros(1, 128), (w[:, None] * v).cumsum(0)])
        l = torch.cat([torch.zeros(1), w.cumsum(0)])
        seen = (torch.arange(nq) + nk - nq + 1).clamp(0, nk) if causal else torch.full((nq,), nk)
        out.append(torch.where(l[seen, None] > 0, upto[seen] * (1.0 / l[seen, None]), 0.0))
        lse.append(l[seen].log())
    return torch.cat(out)[:, None], torch.cat(lse)[:, None]


@pytest.mark.parametrize("by", ["tile", "key"])
@pytest.mark.parametrize("ql,kl,causal", [([2, 70], [140000, 300], False), ([1], [40000], True), ([5, 3], [3, 1000], True), ([300], [5000], True)])
def test_count_bounds(ql, kl, causal, by):
    want = pt.counts(ql, kl, causal, by)
    pt.check_counts(*_counted(ql, kl, causal, by), *want)
    if kl[0] < 1000:
        return
    for at in (0, 128 * (kl[0] // 256), 128 * ((kl[0] - 1) // 128) - (300 if ql[0] == 300 else 0) // 128 * 128):
        for weight in (0.0, 2.0):
            with pytest.raises(AssertionError):
                pt.check_counts(*_counted(ql, kl, causal, by, (at, weight)), *want)


@pytest.mark.parametrize("n", [9000, 40000, 140000])
def test_row_bounds(n):
    p, v = pt.exact_row(n)
    ref = ((p / p.sum()) @ v)[None, None], p.sum().log()[None, None]
    rounded = p.to(torch.bfloat16).double()
    ok = ((rounded / p.sum()) @ v)[None, None], p.float().sum().log()[None, None]
    pt.check_rows(*ok, ref)
    pt.check_rows(ok[0].to(torch.bfloat16), ok[1], ref)
    for at in (0, 128 * (n // 256), 128 * (n // 128 - 1)):
        for weight in (0.0, 2.0):
            w = rounded.clone()
            w[at:at + 128] *= weight
            l = p.clone()
            l[at:at + 128] *= weight
            with pytest.raises(AssertionError):  # the values alone, the sum alone
                pt.check_rows(((w / l.sum()) @ v)[None, None], ref[1], ref)
            with pytest.raises(AssertionError):
                pt.check_rows(ok[0], l.sum().log()[None, None], ref)
