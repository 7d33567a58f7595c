"""Decode over a 4-bit cache with block-table entries outside the cache: the
keys of such blocks are left out, all others count. Bounds as in
test_gpu_decode_q4.py."""
import pytest
import torch

from test_gpu_decode_q4 import check, fa, q4_case, run  # noqa: F401

pytestmark = pytest.mark.gpu


def without(cache, table, lens, b, bad, bs):
    """Request b as one of its own over the keys whose blocks are not in `bad`:
    a cache of one-token blocks."""
    t = torch.tensor([i for i in range(int(lens[b])) if i // bs not in bad], dtype=torch.int64)
    rows = [x[table[b, t // bs].long(), :, t % bs][:, :, None] for x in cache]
    return rows, torch.arange(len(t), dtype=torch.int32)[None], torch.tensor([len(t)], dtype=torch.int32)


@pytest.mark.parametrize("H,Hkv", [(4, 2), (8, 1), (16, 1)])
@pytest.mark.parametrize("d,bs,L,bad", [
    (64, 16, 40, [1]), (128, 16, 400, [20]), (128, 16, 700, [0, 3, 8, 9, 43]), (64, 8, 300, [5, 15, 37]),
    (128, 24, 500, [0, 6, 20]), (128, 64, 1000, [1, 15]), (64, 128, 700, [0, 5]), (128, 256, 600, [1]),
    (128, 3, 40, [1]), (64, 5, 300, [0, 26, 59]), (128, 1, 800, [0, 300, 301, 799]),
])
@pytest.mark.parametrize("S", [1, 2])
def test_keys_of_bad_blocks_are_left_out(fa, H, Hkv, d, bs, L, bad, S):  # noqa: F811
    q, cache, table, lens = q4_case(2, H, Hkv, d, bs, [L, L], seed=9 + L + bs)
    ref, rlse = run(fa, q, cache, table, lens, S)
    wrong = table.clone()
    for i, blk in enumerate(bad):
        wrong[1, blk] = (cache[0].shape[0] + 5, -1, cache[0].shape[0], 1 << 30)[i % 4]
    dev = [t.cuda() for t in (q, *cache, wrong, lens)]
    for _ in range(3):
        o, lse = fa.decode_paged_q4(*dev, n_splits=S)
        assert fa.last_device_error() == 7 and fa.last_device_error() == 0
        assert torch.equal(o[0], ref[0]) and torch.equal(lse[0], rlse[0])   # request 0 has none
        rest, table1, lens1 = without(cache, table, lens, 1, bad, bs)
        check(q[1:], rest, table1, lens1, o[1:], lse[1:], d ** -0.5)


@pytest.mark.parametrize("bs", [16, 3])
def test_no_block_left(fa, bs):  # noqa: F811
    q, cache, table, lens = q4_case(2, 8, 2, 128, bs, [200, 90], seed=4)
    table[1] = -7
    o, lse = fa.decode_paged_q4(q.cuda(), *(t.cuda() for t in cache), table.cuda(), lens.cuda(), n_splits=2)
    assert fa.last_device_error() == 7
    assert bool((o[1] == 0).all()) and bool(torch.isneginf(lse[1]).all()) and bool(o[0].isfinite().all())
