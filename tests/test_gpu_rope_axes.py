"""Rotations with several position axes: bit for bit the one-axis calls over
tables that hold each token's own angles (those are held to the fp64
definitions in test_gpu_qk_norm_rope.py and test_gpu_append_paged.py), and the
fp64 definition itself. Bounds of the latter as derived there: a result is
within half a bf16 step, 2^-8 of its value, plus 2^-17 of its row's largest
magnitude for the fp32 roundings before."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import norm_rope

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def own_tables(cos, sin, pos, axes):
    """Tables with a row for each token, [tokens, pairs], of positions [axes, tokens]."""
    axis = torch.tensor(list(axes), device="cuda")
    rows = pos.long()[axis].t()
    pair = torch.arange(len(axes), device="cuda")
    return cos[rows, pair].contiguous(), sin[rows, pair].contiguous()


CASES = [
    # B, H, Hkv, N, d, sections, in turn, interleaved, norm, a table of positions per batch
    (2, 5, 2, 67, 128, (16, 24, 24), False, False, True, True),
    (2, 5, 2, 67, 128, (24, 20, 20), True, False, True, False),
    (1, 3, 3, 130, 64, (1, 2, 5), False, True, True, True),      # sections that split a lane's four pairs
    (1, 3, 3, 130, 64, (11, 13), False, False, False, False),
    (3, 9, 1, 1, 128, (6, 6, 6, 6), True, True, True, True),     # four axes
    (1, 2, 1, 300, 64, (32,), False, False, True, False),        # one
    (2, 4, 2, 33, 128, (0, 40, 24), False, True, False, True),   # an axis no pair is on
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(fa, case):
    B, H, Hkv, N, d, sections, turn, inter, norm, per_batch = case
    g = torch.Generator().manual_seed(sum(sections) + N)
    rn = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
    axes = fa.rope_axes(sections, turn)
    n_pos, rot = 90, 2 * len(axes)
    cos, sin = fa.rope_tables(n_pos, rot)
    shape = (len(sections), B, N) if per_batch else (len(sections), N)
    pos = torch.randint(0, n_pos, shape, generator=g).to(I32).cuda()
    every = pos.expand(-1, N) if pos.dim() == 2 else pos.reshape(len(sections), B * N)
    ocos, osin = own_tables(cos, sin, every.contiguous(), axes)
    own = torch.arange(B * N if per_batch else N, dtype=I32, device="cuda").view((B, N) if per_batch else (N,))
    qkv = rn(B, N, H + 2 * Hkv, d)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
    kw = dict(q_weight=rn(d), k_weight=rn(d)) if norm else {}
    kw["interleaved"] = inter
    got = fa.qk_norm_rope(q, k, cos, sin, positions=pos, axes=axes, **kw)
    ref = fa.qk_norm_rope(q, k, ocos, osin, positions=own, **kw)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    tok = own.cpu().numpy() if per_batch else np.broadcast_to(own.cpu().numpy(), (B, N))
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for a, x, w in ((got[0], q, kw.get("q_weight")), (got[1], k, kw.get("k_weight"))):
        want = norm_rope(to_f64(x), None if w is None else f64(w), f64(ocos), f64(osin), tok, 1e-6, inter)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * np.abs(want).max(-1, keepdims=True)
        assert np.all(np.abs(to_f64(a) - want) <= tol)
    dq, dk = rn(B, H, N, d), rn(B, Hkv, N, d)
    got = fa.qk_norm_rope_bwd(dq, dk, q, k, cos, sin, positions=pos, axes=axes, **kw)
    ref = fa.qk_norm_rope_bwd(dq, dk, q, k, ocos, osin, positions=own, **kw)
    for a, b in zip(got, ref):
        assert (a is None and b is None) or torch.equal(a, b)
    assert fa.last_device_error() == 0


def append_inputs(fa, T, B, H, Hkv, d, bs, q4, seed, n_cached=130):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, H + 2 * Hkv, d), generator=g).to(BF).cuda()
    mb = n_cached // bs + 1
    nb = B * mb + 2
    table = torch.randperm(nb, generator=g)[:B * mb].view(B, mb).to(I32).cuda()
    slot = torch.randperm(B * n_cached, generator=g)[:T]
    req, pos = (slot // n_cached).to(I32).cuda(), (slot % n_cached).to(I32).cuda()
    if q4:
        cache = [t for _ in "kv" for t in (torch.zeros((nb, Hkv, bs, d // 2), dtype=torch.uint8, device="cuda"),
                                           torch.zeros((nb, Hkv, bs, d // 64, 2), dtype=BF, device="cuda"))]
    else:
        cache = [torch.zeros((nb, Hkv, bs, d), dtype=BF, device="cuda") for _ in "kv"]
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(BF).cuda() for _ in "qk"]
    return g, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], cache, table, pos, req, dict(q=qkv[:, :H], q_weight=w[0], k_weight=w[1])


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("T,B,H,Hkv,d,bs,sections,turn,inter", [
    (100, 3, 5, 2, 128, 16, (16, 24, 24), False, False), (70, 2, 4, 4, 64, 3, (5, 2, 9), True, True),
    (1, 1, 8, 1, 128, 16, (30, 34), False, False), (33, 40, 3, 1, 64, 1, (8, 8, 8, 8), True, False)])
def test_appends(fa, q4, T, B, H, Hkv, d, bs, sections, turn, inter):
    g, k, v, cache, table, pos, req, kw = append_inputs(fa, T, B, H, Hkv, d, bs, q4, T + d)
    entry = fa.append_paged_q4 if q4 else fa.append_paged
    axes = fa.rope_axes(sections, turn)
    cos, sin = fa.rope_tables(77, 2 * len(axes))          # fewer rows than slots
    rope = torch.randint(0, 77, (len(sections), T), generator=g).to(I32).cuda()
    ocos, osin = own_tables(cos, sin, rope, axes)
    other = [t.clone() for t in cache]
    kw["interleaved"] = inter
    got = entry(k, v, *cache, table, pos, req, cos, sin, rope_positions=rope, axes=axes, **kw)
    one = torch.arange(T, dtype=I32, device="cuda")
    ref = entry(k, v, *other, table, pos, req, ocos, osin, rope_positions=one, **kw)
    assert torch.equal(got, ref) and all(torch.equal(a, b) for a, b in zip(cache, other))
    # one axis, positions that are the slots: the plain call
    big = fa.rope_tables(131, 2 * len(axes))
    again = [torch.zeros_like(t) for t in cache]
    for t in other:
        t.zero_()
    got = entry(k, v, *other, table, pos, req, *big, rope_positions=pos, **kw)
    ref = entry(k, v, *again, table, pos, req, *big, **kw)
    assert torch.equal(got, ref) and all(torch.equal(a, b) for a, b in zip(other, again))
    assert fa.last_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_captured_on_another_stream_with_fp32_weights(fa, q4):
    """One graph of an append, a rotation and its gradient; positions and inputs change between replays."""
    T, B, H, Hkv, d, bs = 40, 3, 4, 2, 128, 16
    g, k, v, cache, table, pos, req, kw = append_inputs(fa, T, B, H, Hkv, d, bs, q4, 9)
    kw.update({n: kw[n].float() for n in ("q_weight", "k_weight")})
    weights = dict(q_weight=kw["q_weight"], k_weight=kw["k_weight"])
    append = fa.append_paged_q4 if q4 else fa.append_paged
    axes = fa.rope_axes((24, 20, 20), True)
    cos, sin = fa.rope_tables(50, 128)
    rope = torch.randint(0, 50, (3, T), generator=g).to(I32).cuda()
    x, y = (torch.randn((1, h, T, d), generator=g).to(BF).cuda() for h in (H, Hkv))

    def step(cache):
        out = [append(k, v, *cache, table, pos, req, cos, sin, rope_positions=rope, axes=axes, **kw)]
        out += fa.qk_norm_rope(x, y, cos, sin, positions=rope, axes=axes, **weights)
        out += fa.qk_norm_rope_bwd(out[1], out[2], x, y, cos, sin, positions=rope, axes=axes, **weights)
        return out + list(cache)

    step(cache)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        got = step(cache)
    for _ in range(3):
        rope.copy_(torch.randint(0, 50, (3, T), generator=g))
        k.copy_(torch.randn(k.shape, generator=g))
        other = [t.clone() for t in cache]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(other)):
            assert torch.equal(a, b)
    assert fa.last_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_positions_outside_the_tables(fa, q4):
    T, B, H, Hkv, d, bs = 12, 2, 4, 2, 64, 16
    g, k, v, cache, table, pos, req, kw = append_inputs(fa, T, B, H, Hkv, d, bs, q4, 5)
    entry = fa.append_paged_q4 if q4 else fa.append_paged
    axes = fa.rope_axes((10, 12, 10))
    cos, sin = fa.rope_tables(40, 64)
    rope = torch.randint(0, 40, (3, T), generator=g).to(I32).cuda()
    clean = [t.clone() for t in cache]
    ref = entry(k, v, *clean, table, pos, req, cos, sin, rope_positions=rope, axes=axes, **kw)
    bad = {2: (0, -1), 5: (1, 40), 9: (2, 2 ** 31 - 1)}
    for t, (a, x) in bad.items():
        rope[a, t] = x
    pos2 = pos.clone()
    pos2[7] = -1                                           # padding: its positions are not looked at
    rope[:, 7] = -5
    got = entry(k, v, *cache, table, pos2, req, cos, sin, rope_positions=rope, axes=axes, **kw)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 7
    skipped = sorted([*bad, 7])
    for t in range(T):
        row = [c[table[req[t], pos[t] // bs].long(), :, (pos[t] % bs).long()] for c in cache]
        want = [c[table[req[t], pos[t] // bs].long(), :, (pos[t] % bs).long()] for c in clean]
        if t in skipped:
            assert all(bool((r == 0).all()) for r in row) and bool((got[t] == 0).all())
        else:
            assert all(torch.equal(a, b) for a, b in zip(row, want)) and torch.equal(got[t], ref[t])
    # the training form writes zeros for them
    qn, kn = (x.transpose(0, 1)[None].contiguous() for x in (kw["q"], k))
    qo, ko = fa.qk_norm_rope(qn, kn, cos, sin, positions=rope, axes=axes)
    assert fa.last_device_error() == 7
    for t in range(T):
        assert bool((qo[0, :, t] == 0).all()) == (t in skipped) and bool((ko[0, :, t] == 0).all()) == (t in skipped)
    assert fa.last_device_error() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_a_serving_loop(fa, q4):
    """Append a prompt of text and an image in chunks, attend with each, then
    decode: against attention in 64 bits over what the caches were given."""
    H, Hkv, d, bs, N = 8, 2, 128, 16, 150
    g = torch.Generator().manual_seed(40)
    qkv = torch.randn((N, H + 2 * Hkv, d), generator=g).to(BF).cuda()
    axes = fa.rope_axes((16, 24, 24))
    cos, sin = fa.rope_tables(200, d)
    t = torch.arange(N)
    image = (t >= 20) & (t < 100)                          # one frame of 8 x 10
    rope = torch.stack([torch.where(image, torch.full_like(t, 20), torch.where(t < 20, t, t - 70)),
                        torch.where(image, 20 + (t - 20) // 10, torch.where(t < 20, t, t - 70)),
                        torch.where(image, 20 + (t - 20) % 10, torch.where(t < 20, t, t - 70))]).to(I32).cuda()
    table = torch.randperm(12, generator=g)[:10].view(1, 10).to(I32).cuda()
    if q4:
        cache = [x for _ in "kv" for x in (torch.zeros((12, Hkv, bs, d // 2), dtype=torch.uint8, device="cuda"),
                                           torch.full((12, Hkv, bs, 2, 2), float("nan"), dtype=BF, device="cuda"))]
        append, extend = fa.append_paged_q4, fa.extend_paged_q4
    else:
        cache = [torch.full((12, Hkv, bs, d), float("nan"), dtype=BF, device="cuda") for _ in "kv"]
        append, extend = fa.append_paged, fa.extend_paged
    held = [torch.zeros((N, Hkv, d), dtype=BF, device="cuda") for _ in "kv"]
    i32 = lambda *a: torch.tensor(a, dtype=I32, device="cuda")  # noqa: E731
    outs = []
    for lo, hi in ((0, 64), (64, 131), (131, N)):
        x = qkv[lo:hi]
        n = hi - lo
        pos = torch.arange(lo, hi, dtype=I32, device="cuda")
        kw = dict(requests=torch.zeros_like(pos), cos=cos, sin=sin, q=x[:, :H], rope_positions=rope[:, lo:hi].contiguous(),
                  axes=axes)
        if q4:
            kw |= dict(k_values=held[0][lo:hi], v_values=held[1][lo:hi])
        qn = append(x[:, H:H + Hkv], x[:, H + Hkv:], *cache, table, pos, **kw)
        outs.append(extend(qn, *cache, table, i32(hi), i32(0, n))[0])
    o = torch.cat(outs)
    q, k = fa.qk_norm_rope(qkv[None, :, :H].transpose(1, 2), qkv[None, :, H:H + Hkv].transpose(1, 2), cos, sin,
                           positions=rope, axes=axes)
    kr, vr = (held[0], held[1]) if q4 else (k[0].transpose(0, 1), qkv[:, H + Hkv:])
    ro, _ = fa.fwd(q, kr.transpose(0, 1)[None].contiguous(), vr.transpose(0, 1)[None].contiguous(), causal=True)
    # both round their weights (2^-8 of Σ p |v|, |v| up to 4.5) and their results
    assert (o.float() - ro[0].transpose(0, 1).float()).abs().max() <= 2 * (4.5 + 4.5) * 2.0 ** -8
    dec = (fa.decode_paged_q4 if q4 else fa.decode_paged)(q[0, :, -1][None].contiguous(), *cache, table, i32(N), n_splits=1)[0]
    # 4 bits: a decode step holds the cache's values exactly, the chunk rounded to bf16
    assert (dec[0].float() - o[-1].float()).abs().max() <= 2 * (4.5 + 4.5) * 2.0 ** -8
    assert fa.last_device_error() == 0
