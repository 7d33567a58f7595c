"""decode_paged over a cache whose slots past a request's length hold NaN, as
memory that was never written may: the results are those over a clean cache."""
import pytest
import torch

from test_gpu_decode import fa, paged_case, run_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,bs,lens,S", [(64, 16, [37, 1, 128], 1), (128, 16, [130, 5, 1000], 3),
                                         (128, 128, [129, 300, 127], 2), (64, 8, [9, 64, 250], 2),
                                         (128, 3, [40, 700, 2], 2), (128, 1, [50, 129, 1], 1)])
def test_slots_past_the_length_may_hold_anything(fa, d, bs, lens, S):  # noqa: F811
    q, kc, vc, table, L = paged_case(3, 8, 2, d, bs, lens, seed=bs + d)
    ref = run_case(fa, q, kc, vc, table, L, S, d ** -0.5)
    used = torch.zeros((kc.shape[0], bs), dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        used[table[b, t // bs].long(), t % bs] = True
    dead = ~used[:, None, :].expand(-1, kc.shape[1], -1)
    for fill in (float("nan"), float("inf")):
        kc[dead], vc[dead] = fill, fill
        o, lse = run_case(fa, q, kc, vc, table, L, S, d ** -0.5)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("d", [64, 128])
def test_merge_keeps_nan_rows_nan(fa, d):  # noqa: F811
    g = torch.Generator().manual_seed(d)
    o_parts, lse_parts = torch.randn((3, 8, d), generator=g), torch.randn((3, 8), generator=g)
    clean = fa.attn_merge(o_parts.cuda(), lse_parts.cuda())
    nan, inf = float("nan"), float("inf")
    lse_parts[0, 0] = nan                                          # one part of a row
    lse_parts[:, 1] = torch.tensor([-inf, nan, -inf])              # the only part with keys
    lse_parts[:, 2] = nan
    lse_parts[:, 3] = -inf
    o, lse = fa.attn_merge(o_parts.cuda(), lse_parts.cuda())
    assert bool(o[:3].isnan().all()) and bool(lse[:3].isnan().all())
    assert bool((o[3] == 0).all()) and bool(torch.isneginf(lse[3]))
    assert torch.equal(o[4:], clean[0][4:]) and torch.equal(lse[4:], clean[1][4:])
