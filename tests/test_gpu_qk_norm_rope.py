"""Per-head norms with the position rotation, and their gradient, against the
fp64 definitions.

Bounds. A result is rounded once to bf16: half a step, 2^-8 of its value.
Before that a row's values carry fp32 errors: its sum of d squares and the
reciprocal root (d/16 + 10 roundings of 2^-24 relative), two products, and a
rotation of two products and a sum, fewer than 64 roundings in all, each at
most 2^-24 of the row's largest magnitude m: 2^-18 m.
In the gradient the same roundings stand before the result in both r h and
r n mean(h n): 2^-17 of the larger. A weight gradient sums `rows` products
g n in fp32 within a lane (at most `rows` additions, then under 16 in a
tree), so it is off by at most (rows + 64) 2^-24 Σ |g n| for the sum and n.
g itself is a difference of two products, each and their sum rounded: off by
up to 3 · 2^-24 (|dy_a| + |dy_b|) <= 2^-21 max|dy|, however small g is, which
adds 2^-21 Σ max|dy| |n|."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import norm_rope, norm_rope_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def case(B, H, Hkv, N, d, rot, layout, weights, positions, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if layout == "packed":       # the projection's output, as in a layer
        qkv = rn(B, N, H + 2 * Hkv, d).to(torch.bfloat16).cuda()
        q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
    elif layout == "padded":     # rows 16 bytes further apart than they are long
        q, k = (rn(B, h, N, d + 8).to(torch.bfloat16).cuda()[..., :d] for h in (H, Hkv))
    else:
        q, k = rn(B, H, N, d).to(torch.bfloat16).cuda(), rn(B, Hkv, N, d).to(torch.bfloat16).cuda()
    n_pos = N + 37
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    cos = sin = None
    if rot:
        cos, sin = (torch.from_numpy(f(a)).float().cuda() for f in (np.cos, np.sin))
    qw = kw = None
    if weights is not None:
        qw, kw = ((1 + 0.3 * rn(d)).to(weights).cuda() for _ in range(2))
    pos = None
    if positions == "shared":
        pos = torch.randint(0, n_pos, (N,), generator=g).to(torch.int32).cuda()
    elif positions == "own":
        pos = torch.randint(0, n_pos, (B, N), generator=g).to(torch.int32).cuda()
    return q, k, cos, sin, pos, qw, kw


CASES = [
    # B, H, Hkv, N, d, rot, layout, weights, positions, interleaved
    (1, 1, 1, 1, 64, 64, "plain", torch.bfloat16, None, False),
    (1, 1, 1, 1, 128, 128, "plain", torch.float32, "own", True),
    (2, 4, 2, 33, 128, 128, "packed", torch.bfloat16, None, False),
    (2, 5, 1, 70, 128, 64, "packed", torch.float32, "shared", False),   # half rotated
    (3, 6, 3, 31, 128, 48, "padded", torch.bfloat16, "own", False),     # 3 of 8 chunk pairs
    (1, 7, 7, 129, 64, 32, "packed", torch.bfloat16, "own", True),
    (2, 3, 2, 40, 64, 16, "plain", torch.float32, "shared", False),
    (2, 8, 2, 65, 128, 128, "packed", None, "own", False),              # rotation alone
    (1, 9, 1, 64, 64, 64, "plain", None, None, True),
    (2, 4, 4, 17, 128, 0, "packed", torch.bfloat16, None, False),       # norm alone
    (5, 2, 1, 3, 64, 0, "padded", torch.float32, None, False),
    (4, 12, 12, 1028, 64, 64, "plain", torch.bfloat16, None, False),
    (1, 32, 8, 700, 128, 128, "packed", torch.bfloat16, "own", True),
]


def rows_max(x):
    return np.abs(x).max(axis=-1, keepdims=True)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_forward_and_gradient(fa, c):
    B, H, Hkv, N, d, rot, layout, weights, positions, inter = c
    q, k, cos, sin, pos, qw, kw = case(B, H, Hkv, N, d, rot, layout, weights, positions, seed=17 * N + H)
    before = q.clone(), k.clone()
    got = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    assert fa.last_device_error() == 0
    P = None if pos is None else pos.cpu().numpy()
    for x, y, w in ((q, got[0], qw), (k, got[1], kw)):
        ref = norm_rope(to_f64(x), f64(w), f64(cos), f64(sin), P, 1e-5, inter)
        assert y.is_contiguous()
        err = np.abs(to_f64(y) - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * rows_max(ref) * 2), err.max()
    g = torch.Generator().manual_seed(N)
    dqo = torch.randn((B, H, N, d), generator=g).to(torch.bfloat16).cuda()
    dko = torch.randn((B, Hkv, N, d), generator=g).to(torch.bfloat16).cuda()
    grads = fa.qk_norm_rope_bwd(dqo, dko, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5,
                                interleaved=inter)
    assert fa.last_device_error() == 0
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    again = fa.qk_norm_rope_bwd(dqo, dko, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, eps=1e-5,
                                interleaved=inter)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)
    for dy, x, w, dx, dw in ((dqo, q, qw, grads[0], grads[2]), (dko, k, kw, grads[1], grads[3])):
        args = (f64(cos), f64(sin), P, 1e-5, inter)
        rdx, rdw = norm_rope_bwd(to_f64(dy), to_f64(x), f64(w), *args)
        scale = rows_max(rdx)
        if w is not None:
            back, _ = norm_rope_bwd(to_f64(dy), to_f64(x), None, *args)
            r = 1 / np.sqrt(np.mean(to_f64(x) ** 2, -1, keepdims=True) + 1e-5)
            h, n = back * f64(w), to_f64(x) * r
            scale = rows_max(r * h) + rows_max(r * n) * np.abs(np.mean(h * n, -1, keepdims=True))
            terms = np.abs(back * n).sum(axis=(0, 1, 2))
            rows = B * N * x.shape[1]
            assert dw.dtype == torch.float32
            turned = 2.0 ** -21 * (rows_max(to_f64(dy)) * np.abs(n)).sum(axis=(0, 1, 2))
            assert np.all(np.abs(f64(dw) - rdw) <= (rows + 64) * 2.0 ** -24 * terms + turned)
            # a lane's share is far less than all rows: in practice the sum is far closer
            assert np.linalg.norm(f64(dw) - rdw) <= 2e-6 * np.linalg.norm(terms)
        err = np.abs(to_f64(dx) - rdx)
        assert np.all(err <= 2.0 ** -8 * np.abs(rdx) + 2.0 ** -17 * scale), err.max()


def test_gradient_matches_differences(fa):
    # <dx, u> against a difference of the fp64 definition along u, at the
    # points the kernel got (bf16 inputs are exact in 64 bits). The kernel's
    # dx is off by 2^-8 |dx| at most (plus fp32), so <dx, u> by that times |u|.
    q, k, cos, sin, pos, qw, kw = case(1, 2, 1, 9, 64, 64, "plain", torch.float32, "own", seed=5)
    dqo, dko = torch.randn_like(q.float()).to(torch.bfloat16), torch.randn_like(k.float()).to(torch.bfloat16)
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(dqo, dko, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    rng = np.random.default_rng(0)
    P = pos.cpu().numpy()
    for x, dy, w, dx, dw in ((q, dqo, qw, dq, dqw), (k, dko, kw, dk, dkw)):
        X, DY, W = to_f64(x), to_f64(dy), f64(w)
        f = lambda a, b: float((norm_rope(a, b, f64(cos), f64(sin), P) * DY).sum())  # noqa: E731
        for _ in range(5):
            u = rng.standard_normal(X.shape)
            num = (f(X + 1e-5 * u, W) - f(X - 1e-5 * u, W)) / 2e-5
            DX = to_f64(dx)
            assert abs((DX * u).sum() - num) <= 2.0 ** -7 * np.abs(DX * u).sum() + 1e-4
            u = rng.standard_normal(W.shape)
            num = (f(X, W + 1e-5 * u) - f(X, W - 1e-5 * u)) / 2e-5
            assert abs((f64(dw) * u).sum() - num) <= 1e-4 * np.abs(f64(dw) * u).sum() + 1e-5


def test_strided_outputs_and_in_place(fa):
    q, k, cos, sin, pos, qw, kw = case(2, 4, 2, 50, 128, 128, "packed", torch.bfloat16, "own", seed=6)
    ref = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    # into another packed buffer: nothing beside the rows is touched
    buf = torch.full((2, 50, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, q_out=buf[:, :, :4].transpose(1, 2),
                          k_out=buf[:, :, 4:6].transpose(1, 2))
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]) and bool((buf[:, :, 6:] == 7).all())
    g = [torch.randn_like(x.float()).to(torch.bfloat16) for x in ref]
    gref = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    dbuf = torch.full((2, 50, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw,
                              dq=dbuf[:, :, :4].transpose(1, 2), dk=dbuf[:, :, 4:6].transpose(1, 2))
    for a, b in zip(got, gref):
        assert torch.equal(a, b)
    assert bool((dbuf[:, :, 6:] == 7).all())
    # gradients over their own inputs, outputs over theirs
    dq, dk, _, _ = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, dq=g[0], dk=g[1])
    assert torch.equal(dq, gref[0]) and torch.equal(dk, gref[1])
    fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert fa.last_device_error() == 0


def test_broadcast_input(fa):
    # one key head read as three: rows of stride 0
    q, k, cos, sin, pos, qw, kw = case(2, 3, 1, 20, 64, 64, "plain", torch.bfloat16, None, seed=8)
    wide = fa.qk_norm_rope(q, k.expand(2, 3, 20, 64), cos, sin, q_weight=qw, k_weight=kw)
    one = fa.qk_norm_rope(q, k, cos, sin, q_weight=qw, k_weight=kw)
    assert torch.equal(wide[1], one[1].expand(2, 3, 20, 64)) and torch.equal(wide[0], one[0])


def test_position_outside_the_tables_is_reported_not_read(fa):
    q, k, cos, sin, pos, qw, kw = case(1, 2, 1, 12, 64, 64, "plain", torch.bfloat16, "own", seed=9)
    ref = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    bad = pos.clone()
    bad[0, 3], bad[0, 7] = -1, cos.shape[0]
    got = fa.qk_norm_rope(q, k, cos, sin, positions=bad, q_weight=qw, k_weight=kw)
    assert fa.last_device_error() == 7 and fa.last_device_error() == 0
    good = [i for i in range(12) if i not in (3, 7)]
    for a, b in zip(got, ref):
        assert torch.equal(a[:, :, good], b[:, :, good]) and bool((a[:, :, [3, 7]] == 0).all())
    # the gradient: zero for those tokens, and they add nothing to the weights'
    g = [torch.randn_like(x.float()).to(torch.bfloat16) for x in ref]
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=bad, q_weight=qw, k_weight=kw)
    assert fa.last_device_error() == 7
    assert bool((dq[:, :, [3, 7]] == 0).all()) and bool((dk[:, :, [3, 7]] == 0).all())
    ok = [x[:, :, good].contiguous() for x in (*g, q, k)]
    dq2, dk2, dqw2, dkw2 = fa.qk_norm_rope_bwd(*ok, cos, sin, positions=pos[:, good].contiguous(), q_weight=qw,
                                               k_weight=kw)
    assert torch.equal(dq2, dq[:, :, good]) and torch.equal(dk2, dk[:, :, good])
    torch.testing.assert_close(dqw2, dqw, rtol=1e-5, atol=1e-5)


def test_non_finite_rows_stay_their_own(fa):
    q, k, cos, sin, pos, qw, kw = case(1, 4, 2, 40, 128, 128, "packed", torch.bfloat16, None, seed=10)
    ref = fa.qk_norm_rope(q, k, cos, sin, q_weight=qw, k_weight=kw)
    q2 = q.clone()
    q2[0, 1, 5, 3], q2[0, 2, 6, 0] = float("nan"), float("inf")
    got, gk = fa.qk_norm_rope(q2, k, cos, sin, q_weight=qw, k_weight=kw)
    assert bool(got[0, 1, 5].isnan().all()) and bool(got[0, 2, 6].isnan().any())
    keep = torch.ones(4, 40, dtype=torch.bool)
    keep[1, 5] = keep[2, 6] = False
    assert torch.equal(got[0][keep], ref[0][0][keep]) and torch.equal(gk, ref[1])
    # a zero row with eps: zeros; its gradient is finite
    q3 = q.clone()
    q3[0, 0, 0] = 0
    out, _ = fa.qk_norm_rope(q3, k, cos, sin, q_weight=qw, k_weight=kw)
    assert bool((out[0, 0, 0] == 0).all())
    dq = fa.qk_norm_rope_bwd(torch.ones_like(out), torch.ones_like(gk), q3, k, cos, sin, q_weight=qw, k_weight=kw)[0]
    assert bool(dq.isfinite().all())


def test_other_stream_and_graph(fa):
    q, k, cos, sin, pos, qw, kw = case(2, 4, 2, 200, 128, 128, "packed", torch.bfloat16, "own", seed=11)
    g = [torch.randn((2, h, 200, 128), device="cuda").to(torch.bfloat16) for h in (4, 2)]
    ref = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    gref = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
        grads = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    for t in (*out, *grads):
        t.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*out, *grads), (*ref, *gref)):
        assert torch.equal(a, b)


def test_gradients_that_share_a_workspace_or_run_at_once(fa):
    """One workspace for call after call (the sum of one call's partial rows
    against the next call's writes), then two streams at once with their own."""
    def one(seed):
        q, k, cos, sin, pos, qw, kw = case(2, 4, 2, 700, 128, 128, "packed", torch.bfloat16, "own", seed=seed)
        g = [torch.randn((2, h, 700, 128), device="cuda").to(torch.bfloat16) for h in (4, 2)]
        return lambda **ws: fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, **ws)
    calls = [one(50 + i) for i in range(2)]
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    ws = torch.full((fa.qk_norm_rope_bwd_workspace_bytes(2, 700, 128),), 255, dtype=torch.uint8, device="cuda")
    outs = [calls[i % 2](workspace=ws) for i in range(10)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(10):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(calls[i % 2]())
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        for x, y in zip(out, refs[i % 2]):
            assert torch.equal(x, y)
    assert fa.last_device_error() == 0


def test_offsets_past_32_bits(fa):
    # a packed buffer of more than 2^31 elements: only its last rows are used
    H, d, N = 2, 64, 5
    big = torch.empty((2 ** 31 // (8 * d) + 64, 8, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((N, 8, d), device="cuda").to(torch.bfloat16)
    big[-N:] = rows
    stride = big.shape[0] - N
    view = big.as_strided((2, H, N, d), (stride * 8 * d, d, 8 * d, 1))   # batch 1 starts past 2^31 elements
    big[:N] = rows
    cos, sin = fa.rope_tables(N, d)
    w = torch.ones(d, device="cuda")
    q, k = fa.qk_norm_rope(view, view, cos, sin, q_weight=w, k_weight=w)
    assert torch.equal(q[0], q[1]) and torch.equal(q, k)
    fa.qk_norm_rope(view, view, cos, sin, q_weight=w, k_weight=w, q_out=view, k_out=torch.empty_like(k))
    assert torch.equal(view, q) and fa.last_device_error() == 0


def test_training_step_through_attention(fa):
    """norm and rotation -> fwd -> bwd -> their gradient, as a layer runs
    them, against the fp64 composition of the definitions (attention's own
    tolerance on what passes through it)."""
    from oracle import attention_bwd_gqa, attention_fwd_gqa
    from gpu_helpers import TOL_GRAD, assert_o
    B, H, Hkv, N, d = 1, 4, 2, 150, 64
    q, k, cos, sin, pos, qw, kw = case(B, H, Hkv, N, d, d, "packed", torch.bfloat16, None, seed=12)
    v = torch.randn((B, Hkv, N, d), device="cuda").to(torch.bfloat16)
    do = torch.randn((B, H, N, d), device="cuda").to(torch.bfloat16)
    qr, kr = fa.qk_norm_rope(q, k, cos, sin, q_weight=qw, k_weight=kw)
    o, lse = fa.fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(dqr, dkr, q, k, cos, sin, q_weight=qw, k_weight=kw)
    assert fa.last_device_error() == 0
    rq, rk = (norm_rope(to_f64(x), f64(w), f64(cos), f64(sin)) for x, w in ((q, qw), (k, kw)))
    ro, _ = attention_fwd_gqa(rq, rk, to_f64(v), d ** -0.5, True)
    assert_o(o, ro)
    rdq, rdk, _, _ = attention_bwd_gqa(rq, rk, to_f64(v), to_f64(do), d ** -0.5, True)
    for dy, x, w, dx, dw in ((rdq, q, qw, dq, dqw), (rdk, k, kw, dk, dkw)):
        rdx, rdw = norm_rope_bwd(dy, to_f64(x), f64(w), f64(cos), f64(sin))
        r = 1 / np.sqrt(np.mean(to_f64(x) ** 2, -1).min())
        gain = 2 * r * np.abs(f64(w)).max()   # |dx| per |dy| of the norm: r |w|, and as much for its mean term
        assert np.abs(to_f64(dx) - rdx).max() <= gain * TOL_GRAD + 2.0 ** -8 * np.abs(rdx).max()
        n = np.abs(to_f64(x) * r)
        assert np.all(np.abs(f64(dw) - rdw) <= TOL_GRAD * n.sum(axis=(0, 1, 2)))


def test_prefill_and_append_make_the_same_keys(fa):
    # a prompt's rows from qk_norm_rope and from append_paged are the same bits
    H, Hkv, N, d, bs = 6, 2, 75, 128, 16
    for inter, rot in ((False, 128), (True, 64)):
        q, k, cos, sin, pos, qw, kw = case(1, H, Hkv, N, d, rot, "packed", torch.bfloat16, "own", seed=14)
        qo, ko = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, interleaved=inter)
        mb = cos.shape[0] // bs + 1
        table = torch.randperm(mb, device="cuda").to(torch.int32)[None].contiguous()
        kc, vc = (torch.zeros((mb, Hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        uniq = torch.unique(pos[0], return_inverse=True)[1]
        first = [int((uniq == i).nonzero()[0]) for i in range(int(uniq.max()) + 1)]   # one token a position
        sel = torch.tensor(first, device="cuda")
        kt, qt = k[0].transpose(0, 1)[sel], q[0].transpose(0, 1)[sel]
        p = pos[0][sel].contiguous()
        qa = fa.append_paged(kt, kt, kc, vc, table, p, torch.zeros_like(p), cos, sin, q=qt, q_weight=qw, k_weight=kw,
                             interleaved=inter)
        assert torch.equal(qa, qo[0].transpose(0, 1)[sel])
        got = kc[table[0][(p // bs).long()].long(), :, (p % bs).long()]
        assert torch.equal(got, ko[0].transpose(0, 1)[sel]) and fa.last_device_error() == 0


@pytest.mark.parametrize("B,H,Hkv,N,d", [(64, 3, 1, 1, 128), (1, 128, 128, 3, 64), (3, 33, 17, 5, 128), (1, 1, 1, 4096, 64)])
def test_odd_shapes_against_small_calls(fa, B, H, Hkv, N, d):
    # many heads, many batches, one token: the same bits as head by head
    q, k, cos, sin, pos, qw, kw = case(B, H, Hkv, N, d, d, "packed", torch.float32, "own", seed=15)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    for h in sorted({0, H // 2, H - 1}):
        one, _ = fa.qk_norm_rope(q[:, h:h + 1], k[:, :1], cos, sin, positions=pos, q_weight=qw, k_weight=kw)
        assert torch.equal(one[:, 0], qo[:, h])
    _, one = fa.qk_norm_rope(q[:, :1], k[:, Hkv - 1:], cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    assert torch.equal(one[:, 0], ko[:, Hkv - 1])
    g = [torch.randn_like(x.float()).to(torch.bfloat16) for x in (qo, ko)]
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(*g, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw)
    one = fa.qk_norm_rope_bwd(g[0][:, H - 1:].contiguous(), g[1][:, :1].contiguous(), q[:, H - 1:], k[:, :1], cos, sin,
                              positions=pos, q_weight=qw, k_weight=kw)
    assert torch.equal(one[0][:, 0], dq[:, H - 1]) and torch.equal(one[1][:, 0], dk[:, 0])
    assert bool(dqw.isfinite().all()) and bool(dkw.isfinite().all()) and fa.last_device_error() == 0
