"""extend_paged and extend_paged_q4 against the fp64 attention over the values
that the cache holds (tests/extend_cases.py derives the bounds)."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from extend_cases import BF, check, extend_case, run
from oracle import q4_encode, q4_pack, q4_unpack, q4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


CASES = [
    # H, Hkv, d, block size, new tokens, cached tokens
    (8, 2, 128, 16, [1], [1]),
    (8, 2, 128, 16, [5], [300]),
    (8, 2, 128, 16, [70], [70]),                                 # a prompt from scratch, one item and a bit
    (8, 2, 128, 16, [5, 1, 200, 0, 33], [300, 1, 200, 50, 160]),
    (8, 2, 64, 16, [5, 1, 200, 0, 33], [300, 1, 200, 50, 160]),
    (4, 4, 64, 8, [130, 257, 3], [130, 700, 1000]),              # one head a K/V head
    (4, 4, 128, 128, [129, 1], [640, 128]),
    (2, 1, 128, 64, [500], [513]),
    (10, 2, 128, 32, [60, 7], [333, 90]),                        # 5 heads: 125 of 128 rows
    (7, 1, 64, 16, [19, 100], [19, 130]),
    (16, 1, 128, 16, [9, 40], [1000, 41]),
    (71, 1, 64, 16, [3, 4], [100, 4]),                           # one token a query tile
    (130, 1, 64, 16, [3, 2], [260, 2]),                          # a K/V head's query heads in two tiles
    (8, 2, 128, 3, [5, 1, 200, 0, 33], [300, 1, 200, 50, 160]),  # gathered
    (8, 2, 64, 1, [40, 2], [129, 777]),
    (4, 4, 64, 5, [130, 257, 3], [130, 700, 1000]),
    (8, 2, 128, 48, [40, 2], [129, 777]),
    (8, 2, 128, 200, [40, 2], [129, 777]),
    (8, 2, 128, 24, [1, 1, 1], [4000, 17, 128]),
    (8, 2, 128, 16, [20, 4], [5, 0]),                            # tokens before position 0, nothing cached
    (8, 2, 64, 3, [20, 4], [5, 0]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_oracle(fa, case, causal):
    H, Hkv, d, bs, new, lens = case
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, bs, new, lens, seed=H + d + bs + sum(new))
    o, lse = run(fa, q, (kc, vc), table, L, starts, causal=causal)
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse, causal)


def q4_of(x):
    """Codes and pairs of a bf16 cache (slots of NaN hold pairs of NaN), and the bf16 values read back."""
    codes, pairs = q4_encode(x.float().numpy())
    held = torch.from_numpy(np.nan_to_num(q4_values(codes, pairs))).to(torch.float32).to(BF)
    return torch.from_numpy(q4_pack(codes)), torch.from_numpy(pairs).to(BF), held


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_q4_is_the_bf16_call_over_the_values_read_back(fa, case, causal):
    """Bit for bit: both calls cut their work alike (contexts below a chunk)
    and differ in how a tile reaches shared memory only. Every number here has
    few enough bits for the read-back value to be exact before its rounding."""
    H, Hkv, d, bs, new, lens = case
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, bs, new, lens, seed=H + d + bs + sum(new) + 1)
    (kq, ks, kh), (vq, vs, vh) = q4_of(kc), q4_of(vc)
    o, lse = run(fa, q, (kq, ks, vq, vs), table, L, starts, causal=causal)
    ro, rl = run(fa, q, (kh, vh), table, L, starts, causal=causal)
    assert torch.equal(o, ro) and torch.equal(lse, rl)
    check(q, to_f64(kh), to_f64(vh), table, L, starts, o, lse, causal)


def test_q4_every_code_reads_back_rounded_once(fa):
    """One key a request, value weights 1: o is the read-back value row itself."""
    d, n = 128, 32
    g = torch.Generator().manual_seed(9)
    codes = torch.arange(16).repeat(n * d // 16).view(n, 1, 1, d)
    codes = codes[..., torch.randperm(d, generator=g)]
    pairs = torch.stack([torch.rand((n, 1, 1, 2), generator=g) * 2.0 ** torch.randint(-20, 20, (n, 1, 1, 2), generator=g),
                         torch.randn((n, 1, 1, 2), generator=g) * 2.0 ** torch.randint(-20, 20, (n, 1, 1, 2), generator=g)],
                        -1).to(BF)
    pairs[3, 0, 0, 0, 0] = 0.0
    packed = torch.from_numpy(q4_pack(codes.numpy()))
    ref = q4_values(codes.numpy(), pairs.double().numpy())  # exact in 64 bits
    # nearest bf16 of a 64-bit value, ties to even
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-300))) - 7)
    want = torch.from_numpy(np.rint(ref / step) * step).to(torch.float32)
    table = torch.arange(n, dtype=torch.int32)[:, None].contiguous()
    ones = torch.ones(n, dtype=torch.int32)
    q = torch.zeros((n, 1, d), dtype=BF)
    zero = torch.zeros_like(packed), torch.zeros_like(pairs)
    o, _ = run(fa, q, (*zero, packed, pairs), table, ones, torch.arange(n + 1, dtype=torch.int32))
    assert torch.equal(o[:, 0].float().cpu(), want[:, 0, 0])


@pytest.mark.parametrize("H,Hkv,d,new,lens", [(64, 64, 128, [300, 2], [3000, 700]), (128, 128, 64, [1500, 3], [4500, 4000]),
                                              (64, 64, 128, [2000], [2000]), (64, 64, 128, [700, 1600], [1500, 6000]),
                                              (240, 8, 128, [90], [24000])])
def test_keys_in_chunks(fa, H, Hkv, d, new, lens):
    """So many K/V heads, or so long a context, that a chunk of keys is shorter
    than the context, with a few items a head and many."""
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, 16, new, lens, seed=77)
    o, lse = run(fa, q, (kc, vc), table, L, starts)
    kv = list(range(0, Hkv, Hkv // 4))  # the oracle on some heads
    pick = [h * (H // Hkv) + h % (H // Hkv) for h in kv]
    check(q[:, pick], to_f64(kc[:, kv]), to_f64(vc[:, kv]), table, L, starts, o[:, pick], lse[:, pick])


def test_one_token_is_a_decode_step(fa):
    q, (kc, vc), table, L, starts = extend_case(8, 2, 128, 16, [1] * 4, [1, 127, 128, 1000], seed=3)
    o, lse = run(fa, q, (kc, vc), table, L, starts)
    ro, rl = fa.decode_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), L.cuda(), n_splits=2)
    assert (o.float() - ro.float()).abs().max() <= 2.0 ** -7 and (lse - rl).abs().max() <= 2.0 ** -16


def test_a_prompt_in_chunks_is_the_prompt(fa):
    """Chunk after chunk of a prompt over one cache, against the whole forward."""
    H, Hkv, d, N, bs = 8, 2, 128, 700, 16
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((N, h, d), generator=g).to(BF).cuda() for h in (H, Hkv, Hkv))
    table = torch.randperm(50, generator=g)[:44].view(1, 44).to(torch.int32).cuda()
    kc, vc = (torch.full((50, Hkv, bs, d), float("nan"), dtype=BF, device="cuda") for _ in "kv")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for lo, hi in ((0, 1), (1, 130), (130, 131), (131, 600), (600, 700)):
        pos = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
        fa.append_paged(k[lo:hi], v[lo:hi], kc, vc, table, pos, requests=torch.zeros_like(pos))
        outs.append(fa.extend_paged(q[lo:hi], kc, vc, table, i32(hi), i32(0, hi - lo)))
    o, lse = torch.cat([x[0] for x in outs]), torch.cat([x[1] for x in outs])
    ro, rl = fa.fwd(*(t.transpose(0, 1)[None].contiguous() for t in (q, k, v)), causal=True)
    assert fa.last_device_error() == 0
    assert (o.float() - ro[0].transpose(0, 1).float()).abs().max() <= 2.0 ** -6  # roundings of o and of the weights
    assert (lse - rl[0].t()).abs().max() <= 2.0 ** -16


def test_rows_of_no_request(fa):
    q, caches, table, L, starts = extend_case(4, 2, 64, 16, [5, 3], [40, 3], seed=5, before=7, after=200)
    q[:7] = float("nan")
    q[15:] = float("nan")
    o, lse = run(fa, q, caches, table, L, starts)
    assert bool((o[:7] == 0).all()) and bool((o[15:] == 0).all())
    assert bool(torch.isneginf(lse[:7]).all()) and bool(torch.isneginf(lse[15:]).all())
    out, given = torch.full_like(q, 3.0).cuda(), torch.full((215, 4), 5.0, device="cuda")
    run(fa, q, caches, table, L, starts, out=out, lse=given)
    assert torch.equal(out[7:15], o[7:15]) and torch.equal(given[7:15], lse[7:15])
    assert bool((out[:7] == 3).all()) and bool((out[15:] == 3).all())
    assert bool((given[:7] == 5).all()) and bool((given[15:] == 5).all())


def test_no_tokens_at_all(fa):
    q, caches, table, L, _ = extend_case(4, 2, 64, 16, [3, 4], [40, 3], seed=5)
    o, lse = run(fa, q, caches, table, L, torch.zeros(3, dtype=torch.int32))
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("bs", [16, 3])
def test_peaked_scores(fa, bs):
    """Scores far apart: references are raised and O rescaled."""
    q, (kc, vc), table, L, starts = extend_case(8, 2, 128, bs, [140, 9], [900, 500], seed=12, q_std=8.0)
    o, lse = run(fa, q, (kc, vc), table, L, starts)
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse)


def test_scale_and_infinite_scores(fa):
    q, (kc, vc), table, L, starts = extend_case(4, 2, 64, 16, [40, 2], [200, 60], seed=4)
    o, lse = run(fa, q, (kc, vc), table, L, starts, scale=0.3)
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse, scale=0.3)
    q[3, 1] = float("nan")  # one row; the others keep their values
    o2, lse2 = run(fa, q, (kc, vc), table, L, starts, scale=0.3)
    assert bool(o2[3, 1].isnan().all()) and bool(lse2[3, 1].isnan())
    o2[3, 1], lse2[3, 1] = o[3, 1], lse[3, 1]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_same_bits_again_and_beside_another_call(fa):
    a = extend_case(8, 2, 128, 16, [300, 1, 64], [2000, 800, 64], seed=1)
    b = extend_case(8, 2, 64, 3, [100, 30], [900, 1500], seed=2)
    ref = [run(fa, *x) for x in (a, b)]
    dev = [[t.cuda() for t in (x[0], *x[1], *x[2:])] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in dev]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, x in zip(streams, dev):
            with torch.cuda.stream(s):
                got.append(fa.extend_paged(*x))
        torch.cuda.synchronize()
        for r, o in zip(ref, got):
            assert torch.equal(r[0], o[0]) and torch.equal(r[1], o[1])


def test_a_captured_call_takes_other_lengths(fa):
    H, Hkv, d, bs, T, B = 8, 2, 128, 16, 64, 3
    q, caches, table, L, starts = extend_case(H, Hkv, d, bs, [20, 40, 4], [500, 40, 260], seed=6)
    dev = [t.cuda() for t in (q, *caches, table, L, starts)]
    o, lse = torch.empty_like(dev[0]), torch.empty((T, H), device="cuda")
    fa.extend_paged(*dev, out=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.extend_paged(*dev, out=o, lse=lse)
    for lens, cut in (([500, 40, 260], [0, 20, 60, 64]), ([33, 40, 1], [0, 33, 63, 64]), ([500, 40, 260], [0, 0, 30, 64])):
        dev[4].copy_(torch.tensor(lens, dtype=torch.int32))
        dev[5].copy_(torch.tensor(cut, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ro, rl = fa.extend_paged(*dev)
        assert torch.equal(o, ro) and torch.equal(lse, rl)
    assert fa.last_device_error() == 0


@pytest.mark.parametrize("kind", ["16", "3", "q4"])
def test_bad_blocks_and_starts_are_reported(fa, kind):
    bs = 16 if kind == "q4" else int(kind)
    q, caches, table, L, starts = extend_case(4, 2, 64, bs, [5, 30, 3], [40, 90, 30], seed=5, fill=0.0)
    if kind == "q4":
        caches = [t for c in caches for t in q4_of(c)[:2]]
    ref = run(fa, q, caches, table, L, starts)
    entry = fa.extend_paged_q4 if kind == "q4" else fa.extend_paged
    for bad in (-1, caches[0].shape[0], 2 ** 30):
        worse = table.clone()
        worse[1, 1] = bad
        o, lse = entry(q.cuda(), *(c.cuda() for c in caches), worse.cuda(), L.cuda(), starts.cuda())
        torch.cuda.synchronize()
        assert fa.last_device_error() == 7
        for rows in (slice(0, 5), slice(35, 38)):  # the other requests' rows
            assert torch.equal(o[rows], ref[0][rows]) and torch.equal(lse[rows], ref[1][rows])
    for cut in ([0, 5, 3, 38], [0, 5, 40, 38], [-1, 5, 35, 38]):
        o, _ = entry(q.cuda(), *(c.cuda() for c in caches), table.cuda(), L.cuda(),
                     torch.tensor(cut, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert fa.last_device_error() == 7
    assert fa.last_device_error() == 0


def test_many_requests(fa):
    """More requests than a CTA has threads."""
    g = torch.Generator().manual_seed(31)
    B = 1300
    new = torch.randint(0, 4, (B,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 40, (B,), generator=g))]
    q, (kc, vc), table, L, starts = extend_case(2, 1, 64, 16, new, lens, seed=30)
    o, lse = run(fa, q, (kc, vc), table, L, starts)
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse)


def test_random_shapes(fa):
    g = torch.Generator().manual_seed(99)
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    for i in range(40):
        B, Hkv, d = ri(1, 5), ri(1, 3), 64 * ri(1, 2)
        H = Hkv * ri(1, 9)
        bs = [1, 3, 8, 16, 24, 32, 64, 128][ri(0, 7)]
        new = [ri(0, [4, 40, 400][ri(0, 2)]) for _ in range(B)]
        lens = [n + ri(0, [3, 100, 1500][ri(0, 2)]) for n in new]
        if sum(new) == 0:
            continue
        causal = ri(0, 3) > 0
        q, caches, table, L, starts = extend_case(H, Hkv, d, bs, new, lens, seed=1000 + i)
        if ri(0, 2) == 0:
            (kq, ks, kh), (vq, vs, vh) = (q4_of(c) for c in caches)
            o, lse = run(fa, q, (kq, ks, vq, vs), table, L, starts, causal=causal)
            check(q, to_f64(kh), to_f64(vh), table, L, starts, o, lse, causal)
        else:
            o, lse = run(fa, q, caches, table, L, starts, causal=causal)
            check(q, to_f64(caches[0]), to_f64(caches[1]), table, L, starts, o, lse, causal)
