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

