"""Chunk calls whose starts are out of order or range: the requests that are in
order keep their results, the others are empty."""
import pytest
import torch

from extend_cases import BF, extend_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("H,Hkv,T,length", [(32, 8, 400, 16384), (4, 4, 1281, 61440)])
def test_rows_given_twice_are_worked_on_once(fa, H, Hkv, T, length, q4):
    """Starts that go down and up again, keys in chunks: the workspace has room
    for rows that are given once. What lies behind it is NaN and stays."""
    d, bs, nb = 128, 16, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = rn(T, H, d).to(BF)
    table = torch.randint(0, nb, (3, length // bs), generator=g, device="cuda").to(torch.int32)
    if q4:
        codes = [torch.randint(0, 256, (nb, Hkv, bs, d // 2), generator=g, device="cuda").to(torch.uint8) for _ in "kv"]
        pairs = [(0.3 * rn(nb, Hkv, bs, d // 64, 2)).to(BF) for _ in "kv"]
        entry, cache = fa.extend_paged_q4, (codes[0], pairs[0], codes[1], pairs[1])
    else:
        entry, cache = fa.extend_paged, tuple(rn(nb, Hkv, bs, d).to(BF) for _ in "kv")
    need = fa.extend_workspace_bytes(T, 3, H, Hkv, d, bs, length // bs)
    store = torch.full((need // 4 + (1 << 20),), float("nan"), device="cuda")
    ws = store[:need // 4].view(torch.uint8)
    lens = i32([length] * 3)
    ref = entry(q, *cache, table, lens, i32([0, T, T, T]))
    assert fa.last_device_error() == 0
    o, lse = torch.full_like(q, 3.0), torch.full((T, H), 5.0, device="cuda")
    for starts in ([0, T, 0, T], [0, T, T // 2, T], [0, T, T - 1, T]):
        entry(q, *cache, table, lens, i32(starts), workspace=ws, out=o, lse=lse)
        torch.cuda.synchronize()
        assert fa.last_device_error() == 7
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert bool(store[need // 4:].isnan().all())


def test_requests_in_order_keep_their_rows(fa):
    """Broken numbers among many requests, more than a CTA has threads."""
    B, H, Hkv, d, bs = 1200, 2, 1, 64, 16
    new = [1 + b % 3 for b in range(B)]
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, bs, new, [n + b % 40 for b, n in enumerate(new)], seed=4)
    dev = [t.cuda() for t in (q, kc, vc, table, L)]
    ref = fa.extend_paged(*dev, starts.cuda())
    bad = starts.clone()
    bad[1] = -1            # requests 0 and 1
    bad[600] = 2 ** 31 - 1  # 599 and 600
    bad[900] = bad[890]    # 899 goes down, 900 begins within 890
    gone = {0, 1, 599, 600, 899, 900}
    o, lse = torch.full_like(ref[0], 3.0), torch.full_like(ref[1], 5.0)
    fa.extend_paged(*dev, bad.cuda(), out=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 7
    for b in range(B):
        rows = slice(int(starts[b]), int(starts[b + 1]))
        if b in gone:
            assert bool((o[rows] == 3).all()) and bool((lse[rows] == 5).all()), b
        else:
            assert torch.equal(o[rows], ref[0][rows]) and torch.equal(lse[rows], ref[1][rows]), b


@pytest.mark.parametrize("bs", [16, 3])
@pytest.mark.parametrize("starts", [[0, 5, 3, 38], [0, 5, 40, 38], [-1, 5, 35, 38], [2, 5, 35, 60], [4, 30, 20, 36],
                                    [38, 0, 38, 5], [0, 38, 38, 0], [-1, -1, -1, -1], [39, 39, 39, 39]])
def test_rows_of_requests_taken_for_empty_are_zero(fa, starts, bs):
    """Outputs that the call itself makes: every row is written. Given ones keep those rows."""
    T, H, lens = 38, 4, [40, 90, 30]
    q, caches, table, L, _ = extend_case(H, 2, 64, bs, [5, 30, 3], lens, seed=5, fill=0.0)
    dev = [t.cuda() for t in (q, *caches, table, L)]
    owner, end, broken = [-1] * T, 0, False
    for b in range(3):
        s, e = starts[b], starts[b + 1]
        if s < 0 or e > T or e < s:
            broken = True
        elif e > s:
            if s >= end:
                owner[s:e] = [b] * (e - s)
            end = max(end, e)
    nobody = torch.tensor(owner).cuda() < 0
    assert broken == (starts != sorted(starts) or starts[0] < 0 or starts[-1] > T)
    given, lse_given = torch.full((T, H, 64), 3.0, dtype=BF, device="cuda"), torch.full((T, H), 5.0, device="cuda")
    fa.extend_paged(*dev, i32(starts), out=given, lse=lse_given)
    assert fa.last_device_error() == (7 if broken else 0)
    assert bool((given[nobody] == 3).all()) and bool((lse_given[nobody] == 5).all())
    # what the call makes its outputs of held other numbers before
    o, lse = torch.full_like(given, 7.0), torch.full_like(lse_given, 7.0)
    nb, Hkv, bs, d = caches[0].shape
    need = fa.extend_workspace_bytes(T, 3, H, Hkv, d, bs, table.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dq, dk, dv, dt, dl = dev
    ds = i32(starts)
    args = fa._EXTEND_ARGS.pack(dq.data_ptr(), dk.data_ptr(), 0, dv.data_ptr(), 0, dt.data_ptr(), dl.data_ptr(), ds.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, T, 3, H, Hkv, d, nb, bs, table.shape[1],
                                1, 1, 0.125)
    assert fa.lib().fa_extend_paged(args, torch.cuda.current_stream().cuda_stream) == 0
    assert fa.last_device_error() == (7 if broken else 0)
    assert bool((o[nobody] == 0).all()) and bool(torch.isneginf(lse[nobody]).all())
    assert torch.equal(o[~nobody], given[~nobody]) and torch.equal(lse[~nobody], lse_given[~nobody])


def test_gaps_among_many_requests_are_zero(fa):
    B, H, Hkv, d, bs = 1200, 2, 1, 64, 16
    new = [1 + b % 3 for b in range(B)]
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, bs, new, [n + b % 40 for b, n in enumerate(new)], seed=4,
                                                before=4, after=9)
    dev = [t.cuda() for t in (q, kc, vc, table, L)]
    ref = fa.extend_paged(*dev, starts.cuda())
    bad = starts.clone()
    bad[1], bad[600], bad[900], bad[B] = -1, 2 ** 31 - 1, bad[890], -7
    o, lse = fa.extend_paged(*dev, bad.cuda())
    torch.cuda.synchronize()
    assert fa.last_device_error() == 7
    gone = {0, 1, 599, 600, 899, 900, B - 1}
    for b in range(B):
        rows = slice(int(starts[b]), int(starts[b + 1]))
        if b in gone:
            assert bool((o[rows] == 0).all()) and bool(torch.isneginf(lse[rows]).all()), b
        else:
            assert torch.equal(o[rows], ref[0][rows]) and torch.equal(lse[rows], ref[1][rows]), b
    assert torch.equal(o[:4], ref[0][:4]) and torch.equal(o[-9:], ref[0][-9:]) and bool(torch.isneginf(lse[-9:]).all())
