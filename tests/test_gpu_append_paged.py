"""Appends to a paged cache, in bf16 and in 4 bits, against the fp64
definitions. Bounds as in test_gpu_qk_norm_rope.py: a bf16 result is within
2^-8 of its value plus 2^-17 of its row's largest magnitude; values (not
normed, not rotated) are copied exactly. A value held in 4 bits is within
max(s/2, 2^-9 (|z| + 8 s)) of the row's, plus the same 2^-17."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import append_slots, norm_rope, q4_encode, q4_pack, q4_unpack, q4_values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    """T tokens of B requests: some in a row (prompts), some single, in random
    order, some padding; a random table; caches filled with a pattern."""

    def __init__(self, fa, T, B, H, Hkv, d, bs, rot, norm, seed, q4, pad=0, step=False, packed=True):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.B, self.H, self.Hkv, self.d, self.bs = T, B, H, Hkv, d, bs
        qkv = torch.randn((T, H + 2 * Hkv, d), generator=g).to(BF).cuda()
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        if not packed:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        if step:
            pos, req = rng.integers(0, 300, T), None
        else:
            first = rng.integers(0, 100, B)
            req = np.sort(rng.integers(0, B, T))
            pos = np.array([first[r] + t - np.searchsorted(req, r) for t, r in enumerate(req)])
            order = rng.permutation(T)
            pos, req = pos[order], req[order]
            for t in rng.choice(T, pad, replace=False):
                if rng.random() < 0.5:
                    pos[t] = -1
                else:
                    req[t] = -3
        self.n_pos = int(max(pos.max(), 0)) + 1
        mb = self.n_pos // bs + 1
        self.nb = B * mb + 3
        table = rng.permutation(self.nb)[:B * mb].reshape(B, mb)
        self.table_np, self.pos_np, self.req_np = table, pos, req
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()  # noqa: E731
        self.table, self.pos, self.req = i32(table), i32(pos), None if req is None else i32(req)
        self.cos = self.sin = self.qw = self.kw = None
        if rot:
            self.cos, self.sin = fa.rope_tables(self.n_pos, rot)
        if norm:
            self.qw, self.kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(BF).cuda() for _ in range(2))
        n, dev = self.nb, "cuda"
        if q4:
            self.cache = [t for _ in "kv" for t in
                          (torch.randint(0, 256, (n, Hkv, bs, d // 2), generator=g).to(torch.uint8).to(dev),
                           torch.randn((n, Hkv, bs, d // 64, 2), generator=g).to(BF).to(dev))]
        else:
            self.cache = [torch.randn((n, Hkv, bs, d), generator=g).to(BF).to(dev) for _ in "kv"]
        self.before = [t.clone() for t in self.cache]
        self.q_out = torch.full((T, H, d), 5.0, dtype=BF, device=dev)

    def kwargs(self, inter=False):
        return dict(requests=self.req, cos=self.cos, sin=self.sin, q=self.q, q_weight=self.qw, k_weight=self.kw,
                    eps=1e-5, interleaved=inter, q_out=self.q_out)

    def expected(self, x, w, inter):
        """Rows [T, heads, d] after norm and rotation (any row for padding)."""
        pos = np.clip(self.pos_np, 0, None)[None]
        return norm_rope(to_f64(x).transpose(1, 0, 2)[None], f64(w), f64(self.cos), f64(self.sin), pos, 1e-5,
                         inter)[0].transpose(1, 0, 2)

    def slots(self):
        return append_slots(self.table_np, self.pos_np, self.req_np, self.bs)


def close(got, ref):
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * np.abs(ref).max(-1, keepdims=True)
    assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()


CASES = [
    # T, B, H, Hkv, d, bs, rot, norm, interleaved, padding, one token per request
    (1, 1, 1, 1, 64, 16, 64, True, False, 0, False),
    (1, 3, 8, 2, 128, 16, 128, False, True, 0, True),
    (33, 5, 4, 2, 128, 16, 128, True, False, 4, False),
    (70, 3, 7, 1, 128, 1, 64, True, True, 0, False),
    (64, 64, 32, 8, 128, 16, 128, True, False, 0, True),
    (100, 9, 12, 12, 64, 48, 32, True, False, 11, False),
    (47, 2, 5, 5, 64, 3, 16, False, False, 1, False),
    (40, 4, 6, 3, 128, 64, 48, True, False, 39, False),
    (20, 2, 9, 3, 128, 5, 0, True, False, 0, False),       # norm alone
    (20, 2, 4, 4, 64, 8, 0, False, False, 2, False),       # a plain copy
    (500, 7, 16, 1, 128, 32, 128, True, False, 20, False),
]
ids = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_append_bf16(fa, c):
    T, B, H, Hkv, d, bs, rot, norm, inter, pad, step = c
    s = Case(fa, T, B, H, Hkv, d, bs, rot, norm, seed=T + H + bs, q4=False, pad=pad, step=step)
    out = fa.append_paged(s.k, s.v, *s.cache, s.table, s.pos, **s.kwargs(inter))
    assert out is s.q_out and fa.last_device_error() == 0
    K, Q, V = s.expected(s.k, s.kw, inter), s.expected(s.q, s.qw, inter), to_f64(s.v)
    kc, vc, q = (to_f64(t) for t in (*s.cache, s.q_out))
    written = np.zeros((s.nb, bs), dtype=bool)
    for t, blk, slot in s.slots():
        close(kc[blk, :, slot], K[t])
        close(q[t], Q[t])
        assert np.array_equal(vc[blk, :, slot], V[t])
        written[blk, slot] = True
    rest = torch.from_numpy(~written)
    for now, before in zip(s.cache, s.before):   # every other row as it was
        assert torch.equal(now.transpose(1, 2).cpu()[rest], before.transpose(1, 2).cpu()[rest])
    live = {t for t, _, _ in s.slots()}
    assert all(np.all(q[t] == 5.0) for t in range(T) if t not in live)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_append_q4(fa, c):
    T, B, H, Hkv, d, bs, rot, norm, inter, pad, step = c
    s = Case(fa, T, B, H, Hkv, d, bs, rot, norm, seed=T + H + bs, q4=True, pad=pad, step=step, packed=T % 2 == 0)
    values = [torch.full((T, Hkv, d), 5.0, dtype=BF, device="cuda") for _ in "kv"]
    fa.append_paged_q4(s.k, s.v, *s.cache, s.table, s.pos, k_values=values[0], v_values=values[1], **s.kwargs(inter))
    assert fa.last_device_error() == 0
    K, Q, V = s.expected(s.k, s.kw, inter), s.expected(s.q, s.qw, inter), to_f64(s.v)
    codes = [s.cache[i].cpu().numpy() for i in (0, 2)]
    pairs = [to_f64(s.cache[i]) for i in (1, 3)]
    q = to_f64(s.q_out)
    written = np.zeros((s.nb, bs), dtype=bool)
    for t, blk, slot in s.slots():
        close(q[t], Q[t])
        # values are copied bf16 numbers: their codes are known exactly
        vcodes, vpairs = q4_encode(V[t].astype(np.float32))
        assert np.array_equal(codes[1][blk, :, slot], q4_pack(vcodes))
        assert np.array_equal(pairs[1][blk, :, slot], vpairs)
        # keys: the grid within one bf16 step of the fp64 key's, and every
        # value held within the stated bound of the key
        _, kpairs = q4_encode(K[t].astype(np.float32))
        p = pairs[0][blk, :, slot]
        assert np.all(np.abs(p - kpairs) <= 2.0 ** -7 * np.abs(kpairs) + 2.0 ** -20)
        held = q4_values(q4_unpack(codes[0][blk, :, slot]), p)
        st, z = p[..., 0].repeat(64, -1), np.abs(p[..., 1]).repeat(64, -1)
        bound = np.maximum(st / 2, 2.0 ** -9 * (z + 8 * st)) + 2.0 ** -17 * np.abs(K[t]).max(-1, keepdims=True)
        assert np.all(np.abs(held - K[t]) <= bound)
        for got, c8, pr in ((values[0], codes[0], pairs[0]), (values[1], codes[1], pairs[1])):
            ref = torch.from_numpy(q4_values(q4_unpack(c8[blk, :, slot]), pr[blk, :, slot])).float().to(BF)
            assert torch.equal(got[t].cpu(), ref)
        written[blk, slot] = True
    rest = torch.from_numpy(~written)
    for now, before in zip(s.cache, s.before):
        assert torch.equal(now.transpose(1, 2).cpu()[rest], before.transpose(1, 2).cpu()[rest])
    live = {t for t, _, _ in s.slots()}
    for t in range(T):
        if t not in live:
            assert np.all(q[t] == 5.0) and all(bool((x[t] == 5).all()) for x in values)


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True)])
def test_q4_keys_without_norm_are_exact(fa, rot, inter):
    # rotation alone is products and sums in fp32, each rounded by itself: the
    # codes are those of the same operations on the host. Enough keys that a
    # contracted sum, which moves one group's step in 10^4, would show.
    s = Case(fa, 6000, 3, 1, 8, 128, 16, rot, False, seed=3, q4=True)
    fa.append_paged_q4(s.k, s.v, *s.cache, s.table, s.pos, s.req, s.cos, s.sin, interleaved=inter)
    x = s.k.float().cpu().numpy()
    cos, sin = (t.cpu().numpy()[s.pos_np][:, None] for t in (s.cos, s.sin))
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    slots = s.slots()
    t, blk, slot = (np.array(c) for c in zip(*slots))
    codes, pairs = q4_encode(y)
    vcodes, vpairs = q4_encode(s.v.float().cpu().numpy())
    for c, ref in zip(s.cache, (q4_pack(codes), pairs, q4_pack(vcodes), vpairs)):
        got = c.float().cpu().numpy().transpose(0, 2, 1, *range(3, c.dim()))[blk, slot]
        assert np.array_equal(got, ref[t].astype(np.float32))


def test_q4_odd_groups(fa):
    """Constant, zero, tiny, huge and non-finite groups."""
    d, T = 128, 8
    v = torch.randn((T, 1, d)).float()
    v[0] = 1.5
    v[1] = 0.0
    v[2, 0, 5], v[3, 0, 70], v[4, 0, 127] = float("nan"), float("inf"), float("-inf")
    v[5] *= 2.0 ** -126
    v[6] *= 2.0 ** 120
    v[7, 0, :64] = torch.where(torch.arange(64) % 2 == 0, 3.0e38, -3.0e38)
    v = v.to(BF).cuda()
    k = torch.zeros_like(v)
    cache = [torch.zeros((1, 1, 16, d // 2), dtype=torch.uint8, device="cuda"),
             torch.zeros((1, 1, 16, 2, 2), dtype=BF, device="cuda")]
    cache += [t.clone() for t in cache]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.append_paged_q4(k, v, *cache, i32(0)[None], i32(*range(T)), i32(*[0] * T))
    assert fa.last_device_error() == 0
    codes, pairs = q4_encode(v[:, 0].float().cpu().numpy())
    np.testing.assert_array_equal(cache[2][0, 0, :T].cpu().numpy(), q4_pack(codes))
    np.testing.assert_array_equal(to_f64(cache[3])[0, 0, :T], pairs)
    assert bool((cache[1].float()[0, 0, :T] == 0).all())


@pytest.mark.parametrize("q4", [False, True])
def test_bad_indices_are_reported_not_used(fa, q4):
    s = Case(fa, 12, 3, 2, 2, 64, 4, 64, True, seed=8, q4=q4)
    fn = fa.append_paged_q4 if q4 else fa.append_paged
    pos, req = s.pos_np.copy(), s.req_np.copy()
    table = s.table_np.copy()
    req[2] = 3                                     # no such request
    pos[5] = table.shape[1] * 4                    # past the table
    used = {(int(r), int(p) // 4) for t, (r, p) in enumerate(zip(req, pos)) if t not in (2, 5)}
    hit = [t for t in range(12) if t not in (2, 5)][0]
    table[req[hit], pos[hit] // 4] = s.nb + 7      # no such block
    skipped = {2, 5} | {t for t in range(12) if t not in (2, 5) and
                        (int(req[t]), int(pos[t]) // 4) == (int(req[hit]), int(pos[hit]) // 4)}
    assert used
    i32 = lambda a: torch.from_numpy(a).to(torch.int32).cuda()  # noqa: E731
    kw = s.kwargs()
    kw["requests"] = i32(req)
    fn(s.k, s.v, *s.cache, i32(table), i32(pos), **kw)
    assert fa.last_device_error() == 7 and fa.last_device_error() == 0
    q = to_f64(s.q_out)
    Q = s.expected(s.q, s.qw, False)
    written = np.zeros((s.nb, 4), dtype=bool)
    for t in range(12):
        if t in skipped:
            assert np.all(q[t] == 5.0)
        else:
            close(q[t], Q[t])
            written[table[req[t], pos[t] // 4], pos[t] % 4] = True
    rest = torch.from_numpy(~written)
    for now, before in zip(s.cache, s.before):
        assert torch.equal(now.transpose(1, 2).cpu()[rest], before.transpose(1, 2).cpu()[rest])
    # a position past the rotation tables alone
    kw = s.kwargs()
    kw["cos"], kw["sin"] = s.cos[:1].contiguous(), s.sin[:1].contiguous()
    fn(s.k, s.v, *s.cache, s.table, s.pos, **kw)
    assert fa.last_device_error() == 7


@pytest.mark.parametrize("q4", [False, True])
def test_graph_replays_on_new_inputs(fa, q4):
    """A captured step with padding rows, replayed after the tokens, positions
    and table changed in place."""
    a = Case(fa, 30, 4, 4, 2, 128, 16, 128, True, seed=21, q4=q4, pad=5)
    b = Case(fa, 30, 4, 4, 2, 128, 16, 128, True, seed=22, q4=q4, pad=9)
    fn = fa.append_paged_q4 if q4 else fa.append_paged
    n = max(a.n_pos, b.n_pos)
    a.cos, a.sin = fa.rope_tables(n, 128)
    b.cos, b.sin = a.cos, a.sin
    w = max(a.table.shape[1], b.table.shape[1])
    total = max(a.nb, b.nb)
    qkv = torch.cat([a.q, a.k, a.v], 1)
    table = torch.zeros((4, w), dtype=torch.int32, device="cuda")
    pos, req, out = a.pos.clone(), a.req.clone(), a.q_out
    caches = [torch.zeros((total, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in a.cache]
    qw, kw = a.qw, a.kw

    def step():
        fn(qkv[:, 4:6], qkv[:, 6:], *caches, table, pos, requests=req, cos=a.cos, sin=a.sin, q=qkv[:, :4], q_weight=qw,
           k_weight=kw, q_out=out)

    table[:, :a.table.shape[1]] = a.table
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c in (a, b):
        table.zero_()
        table[:, :c.table.shape[1]] = c.table
        qkv.copy_(torch.cat([c.q, c.k, c.v], 1))
        pos.copy_(c.pos)
        req.copy_(c.req)
        out.fill_(5.0)
        for t in caches:
            t.zero_()
        graph.replay()
        want = [torch.zeros_like(t) for t in caches]
        ref = torch.full_like(out, 5.0)
        fn(c.k, c.v, *want, table, c.pos, requests=c.req, cos=a.cos, sin=a.sin, q=c.q, q_weight=qw, k_weight=kw,
           q_out=ref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and all(torch.equal(x, y) for x, y in zip(caches, want))
    assert fa.last_device_error() == 0


def test_cache_offsets_past_32_bits(fa):
    # a cache of more than 2^32 bytes a tensor; its last block and a low one
    d, Hkv, bs = 128, 8, 16
    nb = 2 ** 31 // (Hkv * bs * d) + 5
    kc = torch.zeros((nb, Hkv, bs, d), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    k, v = (torch.randn((2, Hkv, d), device="cuda").to(BF) for _ in range(2))
    table = torch.tensor([[nb - 1], [3]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([15, 2], dtype=torch.int32, device="cuda")
    fa.append_paged(k, v, kc, vc, table, pos)
    assert torch.equal(kc[nb - 1, :, 15], k[0]) and torch.equal(vc[nb - 1, :, 15], v[0])
    assert torch.equal(kc[3, :, 2], k[1]) and int((kc != 0).any(-1).sum()) == 2 * Hkv
    assert fa.last_device_error() == 0


def test_same_slot_twice_holds_parts_of_either(fa):
    k, v = (torch.randn((2, 1, 64), device="cuda").to(BF) for _ in range(2))
    kc, vc = (torch.zeros((1, 1, 4, 64), dtype=BF, device="cuda") for _ in range(2))
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.append_paged(k, v, kc, vc, i32(0)[None], i32(1, 1), i32(0, 0))
    for got, new in ((kc, k), (vc, v)):
        assert bool(((got[0, :, 1] == new[0]) | (got[0, :, 1] == new[1])).all())
        assert bool((got[0, :, 2:] == 0).all() and (got[0, :, 0] == 0).all())
    assert fa.last_device_error() == 0


def test_prompt_then_steps_with_bf16_decode(fa):
    """A prompt and three decode steps over the bf16 cache, as a server runs
    them, against attention over the definitions' keys in 64 bits."""
    from gpu_helpers import assert_o
    from oracle import decode_paged
    B, H, Hkv, d, bs = 2, 4, 2, 128, 16
    lens = [37, 5]
    T = sum(lens)
    s = Case(fa, T, B, H, Hkv, d, bs, d, True, seed=30, q4=False)
    req = np.repeat(np.arange(B), lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    mb = 4
    rng = np.random.default_rng(0)
    table = rng.permutation(B * mb + 2)[:B * mb].reshape(B, mb)
    i32 = lambda a: torch.from_numpy(np.asarray(a)).to(torch.int32).cuda()  # noqa: E731
    cos, sin = fa.rope_tables(64, d)
    kc, vc = (torch.full((B * mb + 2, Hkv, bs, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    K = np.zeros((B * mb + 2, Hkv, bs, d))
    V = np.zeros_like(K)

    def record(k, v, pos_, req_):
        rows = norm_rope(to_f64(k).transpose(1, 0, 2)[None], f64(s.kw), f64(cos), f64(sin), pos_[None])[0]
        for t in range(len(pos_)):
            K[table[req_[t], pos_[t] // bs], :, pos_[t] % bs] = rows[:, t]
            V[table[req_[t], pos_[t] // bs], :, pos_[t] % bs] = to_f64(v)[t]

    fa.append_paged(s.k, s.v, kc, vc, i32(table), i32(pos), i32(req), cos, sin, k_weight=s.kw)
    record(s.k, s.v, pos, req)
    for _ in range(3):
        qkv = torch.randn((B, H + 2 * Hkv, d), device="cuda").to(BF)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        at = np.array(lens)
        lens = [n + 1 for n in lens]
        qr = fa.append_paged(k, v, kc, vc, i32(table), i32(at), cos=cos, sin=sin, q=q, q_weight=s.qw, k_weight=s.kw)
        o, lse = fa.decode_paged(qr, kc, vc, i32(table), i32(lens), n_splits=2)
        assert fa.last_device_error() == 0
        record(k, v, at, np.arange(B))
        Q = norm_rope(to_f64(q).transpose(1, 0, 2)[None], f64(s.qw), f64(cos), f64(sin), at[None])[0].transpose(1, 0, 2)
        ro, rlse = decode_paged(Q, K, V, table, np.array(lens), d ** -0.5)
        assert_o(o, ro)
        # a score's q and k are rounded to bf16: each is off by 2^-8 of its
        # norm at most, so a scaled score by 2^-7 |q| |k| / sqrt(d)
        norm = lambda x: np.sqrt((x * x).sum(-1)).max()  # noqa: E731
        assert np.abs(f64(lse) - rlse).max() <= 2.0 ** -7 * norm(Q) * norm(K) * d ** -0.5
