"""extend_paged and extend_paged_q4 at the ends of what they index: caches and
outputs past 2^31 elements, lengths past the table, table entries past the
lengths, items in many parts, captured calls over codes on another stream."""
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from extend_cases import BF, check, extend_case
from oracle import q4_encode, q4_pack, q4_unpack, q4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def codes_of(caches):
    """Codes and pairs of bf16 caches (NaN in slots without a token: pairs of NaN)."""
    out = []
    for c in caches:
        codes, pairs = q4_encode(c.float().numpy())
        out += [torch.from_numpy(q4_pack(codes)), torch.from_numpy(pairs).to(BF)]
    return out


def held(codes, pairs):
    return torch.from_numpy(q4_values(q4_unpack(codes.numpy()), to_f64(pairs))).to(torch.float32).to(BF)


@pytest.mark.parametrize("kind", ["16", "5", "q4"])
def test_blocks_past_32_bits(fa, kind):
    """A cache of more than 2^31 elements (and bytes), its used blocks the last ones: bit for bit the small cache's result."""
    bs, d, Hkv = (16 if kind == "q4" else int(kind)), 128, 8
    q, caches, table, L, starts = extend_case(16, Hkv, d, bs, [40, 3, 1], [300, 90, 17], seed=8)
    if kind == "q4":
        caches = codes_of(caches)
    entry = fa.extend_paged_q4 if kind == "q4" else fa.extend_paged
    args = [t.cuda() for t in (table, L, starts)]
    ref = entry(q.cuda(), *(c.cuda() for c in caches), *args)
    used = caches[0].shape[0]
    per_block = caches[0][0].numel()
    far = 2 ** 31 // per_block + 5  # blocks in front
    big = []
    for c in caches:
        t = torch.empty((far + used, *c.shape[1:]), dtype=c.dtype, device="cuda")
        t[far:] = c.cuda()
        big.append(t)
    args[0] = args[0] + far
    o, lse = entry(q.cuda(), *big, *args)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_rows_past_32_bits(fa):
    """More than 2^31 elements of q and o: the first request, the one across that line and the last."""
    H, Hkv, d, bs, n, B = 32, 2, 128, 16, 1024, 514
    _, (kc, vc), table, _, _ = extend_case(H, Hkv, d, bs, [n], [n], seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty((B * n, H, d), dtype=BF, device="cuda").normal_(generator=g)
    assert q.numel() > 2 ** 31 + n * H * d
    L = torch.full((B,), n, dtype=torch.int32)
    starts = torch.arange(B + 1, dtype=torch.int32) * n
    o, lse = fa.extend_paged(q, kc.cuda(), vc.cuda(), table.repeat(B, 1).cuda(), L.cuda(), starts.cuda())
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    for b in (0, 2 ** 31 // (n * H * d) - 1, 2 ** 31 // (n * H * d), B - 1):
        # every eighth head, four query heads' shares of each K/V head
        rows, heads = slice(b * n, (b + 1) * n), slice(0, H, 8)
        check(q[rows, heads].cpu(), to_f64(kc), to_f64(vc), table, L[:1], starts[:2], o[rows, heads], lse[rows, heads])


@pytest.mark.parametrize("kind", ["16", "3", "q4"])
def test_lengths_past_the_table_and_below_zero(fa, kind):
    bs = 16 if kind == "q4" else int(kind)
    q, caches, table, L, starts = extend_case(4, 2, 64, bs, [20, 30, 9], [2 * bs, 5 * bs, 40], seed=5, fill=0.0)
    if kind == "q4":
        caches = codes_of(caches)
    entry = fa.extend_paged_q4 if kind == "q4" else fa.extend_paged
    dev = [t.cuda() for t in (q, *caches, table)]
    room = table.shape[1] * bs
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    ref = entry(*dev, i32(room, 5 * bs, 0), starts.cuda())
    for over in (room + 1, 2 ** 31 - 1):
        got = entry(*dev, i32(over, 5 * bs, -over), starts.cuda())
        torch.cuda.synchronize()
        assert fa.last_device_error() == 0
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert bool((ref[0][50:] == 0).all()) and bool(torch.isneginf(ref[1][50:]).all())


@pytest.mark.parametrize("H,Hkv,d,bs,new,lens", [
    (8, 1, 128, 16, [30], [60000]),                # one item in 90 parts
    (8, 2, 64, 16, [3, 33], [20000, 31000]),       # few rows
    (32, 4, 128, 64, [1], [30000]),                # one token a K/V head
    (12, 2, 128, 5, [43, 1], [9001, 17]),          # gathered; 6 heads, 126 of 128 rows
    (8, 8, 64, 32, [200, 256], [4000, 6000]),      # two full tiles an item, many items
])
def test_items_in_many_parts(fa, H, Hkv, d, bs, new, lens):
    """Items that many shares cut: their rows are joined by all of those shares' blocks."""
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, bs, new, lens, seed=sum(lens))
    o, lse = fa.extend_paged(*(t.cuda() for t in (q, kc, vc, table, L, starts)))
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse)


def test_two_captured_calls_over_codes_on_another_stream(fa):
    """Two graphs with a workspace each, replayed side by side with lengths that change between replays."""
    H, Hkv, d, bs, T = 8, 2, 128, 16, 200
    q, caches, table, L, starts = extend_case(H, Hkv, d, bs, [150, 46, 4], [1500, 46, 700], seed=6, fill=0.0)
    dev = [t.cuda() for t in (q, *codes_of(caches), table, L, starts)]
    dev[7:] = []
    lens, cuts = dev[6], starts.cuda()
    outs, graphs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    fa.extend_paged_q4(*dev[:6], lens, cuts)
    torch.cuda.synchronize()
    for s in streams:
        o, lse = torch.empty_like(dev[0]), torch.empty((T, H), device="cuda")
        ws = torch.empty(fa.extend_workspace_bytes(T, 3, H, Hkv, d, bs, table.shape[1]), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fa.extend_paged_q4(*dev[:6], lens, cuts, workspace=ws, out=o, lse=lse)
        outs.append((o, lse, ws))
        graphs.append(g)
    for n, c in (([1500, 46, 700], [0, 150, 196, 200]), ([33, 40, 1], [0, 33, 199, 200]), ([700, 46, 700], [0, 0, 100, 200])):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        cuts.copy_(torch.tensor(c, dtype=torch.int32))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        ro, rl = fa.extend_paged_q4(*dev[:6], lens, cuts)
        for o, lse, _ in outs:
            assert torch.equal(o, ro) and torch.equal(lse, rl)
    assert fa.last_device_error() == 0
    k, v = held(dev[1].cpu(), dev[2].cpu()), held(dev[3].cpu(), dev[4].cpu())
    check(q, to_f64(k), to_f64(v), table, lens.cpu(), cuts.cpu(), ro, rl)


@pytest.mark.parametrize("kind", ["16", "128", "3", "q4"])
def test_table_entries_past_the_lengths_are_not_read(fa, kind):
    bs = 16 if kind == "q4" else int(kind)
    q, caches, table, L, starts = extend_case(8, 2, 128, bs, [9, 140, 1], [130, 517, 1], seed=2, fill=0.0)
    if kind == "q4":
        caches = codes_of(caches)
    entry = fa.extend_paged_q4 if kind == "q4" else fa.extend_paged
    dev = [t.cuda() for t in (q, *caches)]
    ref = entry(*dev, table.cuda(), L.cuda(), starts.cuda())
    past = torch.arange(table.shape[1])[None] * bs >= L[:, None]
    assert bool(past.any())
    for junk in (-1, 2 ** 31 - 1):
        got = entry(*dev, table.masked_fill(past, junk).cuda(), L.cuda(), starts.cuda())
        torch.cuda.synchronize()
        assert fa.last_device_error() == 0
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (17, 1), (33, 1), (100, 2), (257, 1)])
def test_head_groups(fa, H, Hkv, d):
    q, (kc, vc), table, L, starts = extend_case(H, Hkv, d, 16, [1, 13, 70], [1, 200, 333], seed=H + d)
    o, lse = fa.extend_paged(*(t.cuda() for t in (q, kc, vc, table, L, starts)))
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    check(q, to_f64(kc), to_f64(vc), table, L, starts, o, lse)
