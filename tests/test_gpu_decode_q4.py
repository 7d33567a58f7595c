"""Decode over a cache held in 4 bits, against the fp64 decode over the values
that its codes stand for.

Bounds. With p the softmax's weights (Σ p = 1) and v = z + s (n − 8), the
kernel rounds each p s to bf16 (2^-8 relative) before the product with n − 8:
at most 2^-8 Σ p |s (n − 8)|. The result is rounded to bf16 once: 2^-8 |o|.
Scores are fp32 sums of at most 128 products |q (n − 8)| <= 8 |q|, scaled by
s, under 2^7 roundings of 2^-24 (twice that where the tensor core truncates):
a score is off by at most e = 2^-14 Σ|q| s · scale in natural units, so p by
2 e and o by 2 e max|v|; lse by e plus the logarithm's 2^-20."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import decode_paged, q4_unpack, q4_values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def q4_case(B, H, Hkv, d, bs, lens, seed, q_std=1.0, offset=0.0, garbage=True):
    """q and a cache whose blocks are placed at random; slots without a token
    hold codes of NaN."""
    g = torch.Generator().manual_seed(seed)
    nb = [(n + bs - 1) // bs for n in lens]
    total = sum(nb) + 3
    q = (torch.randn((B, H, d), generator=g) * q_std).to(BF)
    perm = torch.randperm(total, generator=g)
    table = torch.zeros((B, max(max(nb), 1)), dtype=torch.int32)
    used = torch.zeros((total, bs), dtype=torch.bool)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]].to(torch.int32)
        t = torch.arange(lens[b])
        used[perm[at:at + nb[b]][t // bs], t % bs] = True
        at += nb[b]
    cache = []
    for _ in "kv":
        codes = torch.randint(0, 256, (total, Hkv, bs, d // 2), generator=g).to(torch.uint8)
        pairs = torch.stack([torch.rand((total, Hkv, bs, d // 64), generator=g) * 0.4 + 0.1,
                             torch.randn((total, Hkv, bs, d // 64), generator=g) * 0.3 + offset], -1).to(BF)
        if garbage:
            pairs[~used[:, None, :].expand(total, Hkv, bs)] = float("nan")
        cache += [codes, pairs]
    return q, cache, table, torch.tensor(lens, dtype=torch.int32)


def run(fa, q, cache, table, lens, S, **kw):
    o, lse = fa.decode_paged_q4(q.cuda(), *(t.cuda() for t in cache), table.cuda(), lens.cuda(), n_splits=S, **kw)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    return o, lse


def check(q, cache, table, lens, o, lse, scale):
    Q, L = to_f64(q), lens.numpy()
    kp, vp = np.nan_to_num(to_f64(cache[1])), np.nan_to_num(to_f64(cache[3]))
    K = q4_values(q4_unpack(cache[0].numpy()), kp)
    vn = q4_unpack(cache[2].numpy())
    V = q4_values(vn, vp)
    spread = np.abs(q4_values(vn, np.stack([vp[..., 0], np.zeros_like(vp[..., 1])], -1)))
    ro, rlse = decode_paged(Q, K, V, table.numpy(), L, scale)
    around, _ = decode_paged(Q, K, spread, table.numpy(), L, scale)
    e = 2.0 ** -14 * np.abs(Q).sum(-1) * kp[..., 0].max() * scale          # [B, H]
    tol = 2.0 ** -8 * (around + np.abs(ro)) * 1.01 + 2 * e[..., None] * np.abs(V).max()
    live = L > 0
    err = np.abs(to_f64(o) - ro)[live]
    assert np.all(err <= tol[live]), (err - tol[live]).max()
    dl = np.abs(lse.double().cpu().numpy()[live] - rlse[live])
    assert np.all(dl <= e[live] + 2.0 ** -20 * (np.abs(rlse[live]) + 1)), dl.max()
    if not live.all():
        dead = torch.from_numpy(~live)
        assert bool((o.cpu()[dead] == 0).all()) and bool(torch.isneginf(lse.cpu()[dead]).all())
    # beside the worst case: the whole result, as a 2-norm
    if live.any():
        assert np.linalg.norm((to_f64(o) - ro)[live]) <= 5e-3 * np.linalg.norm(np.abs(ro[live]) + around[live])


CASES = [
    # B, H, Hkv, d, bs, lens, n_splits (0: the library's)
    (1, 1, 1, 64, 16, [1], 1),
    (1, 8, 1, 128, 16, [16], 1),
    (3, 4, 4, 64, 16, [1, 17, 100], 1),
    (3, 8, 2, 128, 16, [1, 64, 1000], 4),
    (2, 8, 1, 128, 32, [5000, 333], 8),
    (2, 4, 2, 64, 1, [50, 7], 2),
    (2, 32, 8, 128, 128, [4097, 256], 3),
    (1, 16, 1, 128, 16, [777], 5),            # 16 query heads on one K/V head
    (3, 4, 2, 128, 16, [0, 1, 129], 2),       # an empty context
    (3, 8, 2, 128, 16, [0, 300, 5], 1),
    (2, 8, 2, 64, 3, [0, 1000], 1),
    (1, 2, 1, 64, 48, [2000], 7),
    (2, 32, 1, 128, 16, [300, 1500], 3),      # 32 = two times 16
    (1, 24, 1, 64, 32, [777], 2),             # 24 = 16 + 8
    (1, 9, 1, 128, 8, [130], 1),              # one more than eight
    (2, 17, 1, 128, 16, [65, 31], 2),
    (2, 12, 3, 128, 64, [700, 129], 3),
    (2, 16, 2, 128, 3, [700, 131], 2),
    (1, 4, 1, 128, 200, [1000], 2),           # blocks larger than any tile
    (1, 4, 1, 128, 1, [3000], 1),
    (2, 4, 2, 128, 16, [40, 15], 16),         # more splits than tiles
    (2, 8, 2, 64, 7, [2001, 64], 0),
    (1, 7, 7, 128, 16, [20011], 0),
    (5, 12, 12, 64, 16, [0, 699, 1, 16, 333], 0),
]


@pytest.mark.parametrize("c", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_decode_q4_vs_oracle(fa, c):
    B, H, Hkv, d, bs, lens, S = c
    q, cache, table, L = q4_case(B, H, Hkv, d, bs, lens, seed=B * 100 + H + bs + sum(lens))
    o, lse = run(fa, q, cache, table, L, S)
    check(q, cache, table, L, o, lse, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [1, 3])
def test_peaked_scores_raise_the_reference(fa, d, S):
    # scores of a standard deviation near 15 in log2 units: the running
    # maximum keeps outgrowing its reference
    q, cache, table, L = q4_case(2, 16, 2, d, 16, [1500, 700], seed=31 + d, q_std=8.0)
    o, lse = run(fa, q, cache, table, L, S)
    check(q, cache, table, L, o, lse, d ** -0.5)


def test_offset_values(fa):
    # values and keys far from zero: the centres carry them, and the codes'
    # rounding stays that of the spread
    q, cache, table, L = q4_case(2, 8, 2, 128, 16, [900, 40], seed=5, offset=20.0, q_std=0.2)
    o, lse = run(fa, q, cache, table, L, 2, scale=0.05)
    check(q, cache, table, L, o, lse, 0.05)


def test_long_context_sums(fa):
    # a context of 200k tokens on one head: sums over many keys
    q, cache, table, L = q4_case(1, 4, 1, 64, 64, [200_003], seed=6)
    for S in (1, 0):
        o, lse = run(fa, q, cache, table, L, S)
        check(q, cache, table, L, o, lse, 64 ** -0.5)


def test_split_count_does_not_change_the_result(fa):
    q, cache, table, L = q4_case(4, 8, 2, 128, 16, [3000, 10, 640, 2049], seed=7)
    outs = [run(fa, q, cache, table, L, S) for S in (1, 2, 7, 40)]
    for o, lse in outs[1:]:
        assert (o.float() - outs[0][0].float()).abs().max() <= 2e-2
        assert (lse - outs[0][1]).abs().max() <= 1e-4


def test_same_call_twice_gives_the_same_bits(fa):
    q, cache, table, L = q4_case(3, 8, 2, 128, 16, [3000, 10, 640], seed=8)
    a, b = run(fa, q, cache, table, L, 5), run(fa, q, cache, table, L, 5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,bs,L,bad", [(64, 16, 40, 1), (128, 16, 400, 20), (128, 3, 40, 1), (128, 1, 800, 300)])
def test_bad_block_index_is_reported_not_read(fa, d, bs, L, bad):
    q, cache, table, lens = q4_case(2, 4, 2, d, bs, [L, L], seed=9)
    wrong = table.clone()
    wrong[1, bad] = cache[0].shape[0] + 5
    dev = [t.cuda() for t in cache]
    o, _ = fa.decode_paged_q4(q.cuda(), *dev, wrong.cuda(), lens.cuda(), n_splits=2)
    assert fa.last_device_error() == 7 and fa.last_device_error() == 0
    ref, _ = run(fa, q, cache, table, lens, 2)
    assert torch.equal(o[0], ref[0])      # request 0 does not use the bad entry
    wrong[1, bad] = -1
    fa.decode_paged_q4(q.cuda(), *dev, wrong.cuda(), lens.cuda(), n_splits=2)
    assert fa.last_device_error() == 7


def test_lengths_outside_the_table_are_clamped(fa):
    q, cache, table, lens = q4_case(2, 4, 2, 128, 16, [160, 160], seed=10)
    ref = run(fa, q, cache, table, lens, 2)
    got = run(fa, q, cache, table, torch.tensor([160, 1 << 30], dtype=torch.int32), 2)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    o, lse = run(fa, q, cache, table, torch.tensor([-4, 160], dtype=torch.int32), 2)
    assert bool((o[0] == 0).all()) and bool(torch.isneginf(lse[0]).all()) and torch.equal(o[1], ref[0][1])


@pytest.mark.parametrize("S", [1, 3])
def test_non_finite_cached_values_stay_in_their_request_and_head(fa, S):
    q, cache, table, lens = q4_case(2, 4, 2, 128, 16, [100, 90], seed=11)
    ref, rlse = run(fa, q, cache, table, lens, S)
    bad = [t.clone() for t in cache]
    bad[1][table[0, 2], 0, 5] = float("nan")     # a key of request 0, K/V head 0 (query heads 0, 1)
    bad[3][table[1, 1], 1, 3, 1] = float("nan")  # half a value of request 1, K/V head 1 (query heads 2, 3)
    o, lse = run(fa, q, bad, table, lens, S)
    assert bool(o[0, :2].isnan().all()) and bool(lse[0, :2].isnan().all())
    assert torch.equal(o[0, 2:], ref[0, 2:]) and torch.equal(o[1, :2], ref[1, :2])
    assert bool(o[1, 2:, 64:].isnan().all()) and bool(o[1, 2:, :64].isfinite().all())
    assert torch.equal(lse[1], rlse[1])
    # every key NaN, alone in its split
    bad = [t.clone() for t in cache]
    bad[1][:] = float("nan")
    o, lse = run(fa, q, bad, table, lens, S)
    assert bool(o.isnan().all()) and bool(lse.isnan().all())


def test_streams_graphs_and_given_buffers(fa):
    q, cache, table, lens = q4_case(3, 8, 2, 128, 16, [500, 3, 900], seed=12)
    ref = run(fa, q, cache, table, lens, 4)
    dev = [t.cuda() for t in (q, *cache, table, lens)]
    ws = torch.full((fa.decode_workspace_bytes(3, 8, 128, 4),), 255, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fa.decode_paged_q4(*dev, n_splits=4, workspace=ws, out=out, lse=lse)
        s.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        with torch.cuda.graph(graph, stream=s):
            fa.decode_paged_q4(*dev, n_splits=4, workspace=ws, out=out, lse=lse)
    # lengths change between replays; workspace content is ignored
    dev[6].copy_(torch.tensor([20, 600, 0], dtype=torch.int32))
    table2 = table.clone()
    table2[1] = table[2]
    dev[5].copy_(table2)
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    want = run(fa, q, cache, table2, torch.tensor([20, 600, 0], dtype=torch.int32), 4)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and fa.last_device_error() == 0


def test_two_streams_at_once(fa):
    cases = [q4_case(2, 8, 2, 128, 16, [3000 + 900 * i, 77], seed=40 + i) for i in range(2)]
    refs = [run(fa, *c, 6) for c in ((c[0], c[1], c[2], c[3]) for c in cases)]
    dev = [[t.cuda() for t in (c[0], *c[1], c[2], c[3])] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for st, args in zip(streams, dev):
            with torch.cuda.stream(st):
                outs.append(fa.decode_paged_q4(*args, n_splits=6))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, refs[i % 2][0]) and torch.equal(lse, refs[i % 2][1])


def test_cache_offsets_past_32_bits(fa):
    # codes past 4 GiB: a request whose blocks lie at the end of the cache
    d, Hkv, bs = 128, 8, 64
    nb = 2 ** 32 // (Hkv * bs * d // 2) + 40
    q, cache, table, lens = q4_case(1, 8, Hkv, d, bs, [1000], seed=13)
    ref = run(fa, q, cache, table, lens, 2)
    big = []
    n = cache[0].shape[0]
    for t in cache:
        x = torch.zeros((nb, *t.shape[1:]), dtype=t.dtype, device="cuda")
        x[-n:] = t.cuda()
        big.append(x)
    o, lse = fa.decode_paged_q4(q.cuda(), *big, (table + nb - n).cuda(), lens.cuda(), n_splits=2)
    assert fa.last_device_error() == 0
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_prompt_then_steps_over_the_q4_cache(fa):
    """Prompts and decode steps with append_paged_q4 and decode_paged_q4, as a
    server runs them. The held values that the appends give back are what each
    step attends to, so every step is checked against them in 64 bits; beside
    that, the first step is near attention over the unquantised cache."""
    B, H, Hkv, d, bs, mb = 3, 8, 2, 128, 16, 5
    lens = [37, 5, 60]
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.randperm(B * mb + 2, generator=g, device="cuda")[:B * mb].view(B, mb).to(torch.int32)
    cos, sin = fa.rope_tables(bs * mb, d)
    qw, kw = (1 + 0.2 * rn(d).float()).to(BF), (1 + 0.2 * rn(d).float()).to(BF)
    cache = [t for _ in "kv" for t in (torch.randint(0, 256, (B * mb + 2, Hkv, bs, d // 2), device="cuda").to(torch.uint8),
                                       torch.full((B * mb + 2, Hkv, bs, d // 64, 2), float("nan"), dtype=BF, device="cuda"))]
    dense = [torch.zeros((B * mb + 2, Hkv, bs, d), dtype=BF, device="cuda") for _ in "kv"]

    def append(qkv, pos, req):
        T = qkv.shape[0]
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        held = [torch.empty((T, Hkv, d), dtype=BF, device="cuda") for _ in "kv"]
        out = fa.append_paged_q4(k, v, *cache, table, pos, req, cos, sin, q=q, q_weight=qw, k_weight=kw,
                                 k_values=held[0], v_values=held[1])
        fa.append_paged(k, v, *dense, table, pos, req, cos, sin, k_weight=kw)
        return out

    append(rn(sum(lens), H + 2 * Hkv, d), i32([p for n in lens for p in range(n)]),
           i32([r for r, n in enumerate(lens) for _ in range(n)]))
    for _ in range(3):
        q = append(rn(B, H + 2 * Hkv, d), i32(lens), None)
        lens = [n + 1 for n in lens]
        o, lse = fa.decode_paged_q4(q, *cache, table, i32(lens))
        ob, _ = fa.decode_paged(q, *dense, table, i32(lens), n_splits=2)
        assert fa.last_device_error() == 0
        check(q.cpu(), [t.cpu() for t in cache], table.cpu(), torch.tensor(lens, dtype=torch.int32), o, lse, d ** -0.5)
        # 16 levels over about ±2.5 standard deviations: steps of 0.3, errors of 0.1
        assert float((o.float() - ob.float()).pow(2).mean().sqrt()) < 0.15 * float(ob.float().pow(2).mean().sqrt()) + 0.05
