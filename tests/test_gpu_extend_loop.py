"""Appends with position axes and chunk attention together, in 64 bits: queries
and keys against the rotation's definition, each chunk against attention over
what the cache holds (bounds: extend_cases.check; rotations as in
test_gpu_rope_axes.py, half a bf16 step and 2^-17 of a row's largest magnitude
for the fp32 roundings before). And scores that are infinite."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from extend_cases import BF, check, extend_case
from oracle import norm_rope, q4_unpack, q4_values

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("q4", [False, True])
def test_two_requests_chunk_by_chunk(fa, q4, bs):
    H, Hkv, d, sizes = 8, 2, 128, (150, 90)
    g = torch.Generator().manual_seed(41)
    axes = fa.rope_axes((16, 24, 24))
    cos, sin = fa.rope_tables(200, d)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(BF).cuda() for _ in "qk"]
    qkv = [torch.randn((n, H + 2 * Hkv, d), generator=g).to(BF).cuda() for n in sizes]
    rope = [torch.randint(0, 200, (3, n), generator=g).to(I32).cuda() for n in sizes]
    per = -(-max(sizes) // bs)
    nb = 2 * per + 3
    table = torch.randperm(nb, generator=g)[:2 * per].view(2, per).to(I32).cuda()
    nan = float("nan")
    if q4:
        cache = [x for _ in "kv" for x in (torch.zeros((nb, Hkv, bs, d // 2), dtype=torch.uint8, device="cuda"),
                                           torch.full((nb, Hkv, bs, 2, 2), nan, dtype=BF, device="cuda"))]
        append, extend = fa.append_paged_q4, fa.extend_paged_q4
    else:
        cache = [torch.full((nb, Hkv, bs, d), nan, dtype=BF, device="cuda") for _ in "kv"]
        append, extend = fa.append_paged, fa.extend_paged
    i32 = lambda *a: torch.tensor(a, dtype=I32, device="cuda")  # noqa: E731
    spans = (((0, 64), (0, 1)), ((64, 131), (1, 90)), ((131, 150), (90, 90)))
    queries = [[], []]
    for step in spans:
        x = torch.cat([qkv[b][lo:hi] for b, (lo, hi) in enumerate(step)])
        pos = torch.cat([torch.arange(lo, hi, dtype=I32) for lo, hi in step]).cuda()
        req = torch.cat([torch.full((hi - lo,), b, dtype=I32) for b, (lo, hi) in enumerate(step)]).cuda()
        rp = torch.cat([rope[b][:, lo:hi] for b, (lo, hi) in enumerate(step)], 1).contiguous()
        qn = append(x[:, H:H + Hkv], x[:, H + Hkv:], *cache, table, pos, req, cos, sin, q=x[:, :H], q_weight=w[0],
                    k_weight=w[1], rope_positions=rp, axes=axes)
        lens, starts = i32(*(hi for _, hi in step)), i32(0, step[0][1] - step[0][0], len(x))
        o, lse = extend(qn, *cache, table, lens, starts)
        torch.cuda.synchronize()
        assert fa.last_device_error() == 0
        if q4:
            held = [torch.from_numpy(q4_values(q4_unpack(c.cpu().numpy()), to_f64(s))).to(torch.float32).to(BF)
                    for c, s in ((cache[0], cache[1]), (cache[2], cache[3]))]
        else:
            held = cache
        check(qn, *(to_f64(c) for c in held), table.cpu(), lens.cpu(), starts.cpu(), o, lse)
        for b in (0, 1):
            queries[b].append(qn[starts[b]:starts[b + 1]])
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    pair, axis = np.arange(d // 2), np.array(list(axes))
    for b, n in enumerate(sizes):
        rows = rope[b].cpu().numpy()[axis].T  # [n, pairs]
        own = f64(cos)[rows, pair], f64(sin)[rows, pair]
        at = table[b].cpu().long()
        slots = lambda t: t.cpu()[at].transpose(1, 2).flatten(0, 1)[:n]  # noqa: E731
        found = [(torch.cat(queries[b]), qkv[b][:, :H], w[0])]
        if q4:
            assert torch.equal(slots(held[1]).float().isnan(), torch.zeros((n, Hkv, d), dtype=torch.bool))
        else:
            found.append((slots(cache[0]), qkv[b][:, H:H + Hkv], w[1]))
            assert torch.equal(slots(cache[1]), qkv[b][:, H + Hkv:].cpu())
        for got, x, wt in found:
            want = norm_rope(to_f64(x).transpose(1, 0, 2)[None], f64(wt), *own, np.arange(n), 1e-6, False)[0].transpose(1, 0, 2)
            tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * np.abs(want).max(-1, keepdims=True)
            assert np.all(np.abs(to_f64(got) - want) <= tol)


@pytest.mark.parametrize("bs", [16, 3])
def test_keys_at_minus_infinity_weigh_nothing(fa, bs):
    """A key whose score is -inf counts as one that is not there; a token that
    sees no other has o = 0, lse = -inf."""
    q, (kc, vc), table, L, starts = extend_case(4, 2, 64, bs, [200, 3], [320, 3], seed=14, fill=0.0)
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    gone = torch.rand((kc.shape[0], bs), generator=torch.Generator().manual_seed(1)) < 0.3
    first = table[1, :1].long()
    gone[first, :2] = True    # all that request 1's first two tokens see
    if bs >= 3:
        gone[first, 2] = False
    clean = kc.clone()
    kc[:, :, :, 0] = torch.where(gone[:, None], float("-inf"), kc[:, :, :, 0].float()).to(BF)
    o, lse = fa.extend_paged(*(t.cuda() for t in (q, kc, vc, table, L, starts)))
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    # the same by its definition: scores over the finite keys with the others taken out, as -inf
    scale = 64 ** -0.5
    got_o, got_l = to_f64(o), lse.double().cpu().numpy()
    for b, length in enumerate(L.tolist()):
        t = np.arange(length)
        at = table[b].numpy()[t // bs]
        K, V, off = to_f64(clean)[at, :, t % bs], to_f64(vc)[at, :, t % bs], gone.numpy()[at, t % bs]
        lo, hi = starts[b].item(), starts[b + 1].item()
        for i in range(lo, hi):
            seen = (t <= length - (hi - lo) + i - lo) & ~off
            for h in range(4):
                k, v, x = K[:, h // 2], V[:, h // 2], to_f64(q)[i, h]
                if not seen.any():
                    assert np.all(got_o[i, h] == 0) and np.isneginf(got_l[i, h])
                    continue
                s = scale * (k[seen] @ x)
                ref = np.log(np.exp(s - s.max()).sum()) + s.max()
                p = np.exp(s - ref)
                ro, around = p @ v[seen], p @ np.abs(v[seen])
                e = 2.0 ** -16 * np.abs(k).max() * np.abs(x).sum() * scale
                assert abs(got_l[i, h] - ref) <= e + 2.0 ** -20 * (abs(ref) + 1), (i, h)
                tol = (2.0 ** -8 * (around + np.abs(ro)) + 2 * e * around) * 1.01
                assert np.all(np.abs(got_o[i, h] - ro) <= tol), (i, h)


def test_a_row_of_plus_infinity_keeps_to_itself(fa):
    """Scores of +inf and -inf in one row: NaN there, and every other row its bits."""
    q, (kc, vc), table, L, starts = extend_case(4, 2, 64, 16, [40, 2], [200, 60], seed=4)
    dev = [t.cuda() for t in (kc, vc, table, L, starts)]
    o, lse = fa.extend_paged(q.cuda(), *dev)
    q[3, 1, 0] = float("inf")
    o2, lse2 = fa.extend_paged(q.cuda(), *dev)
    assert bool(o2[3, 1].isnan().all()) and bool(lse2[3, 1].isnan())
    o2[3, 1], lse2[3, 1] = o[3, 1], lse[3, 1]
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and fa.last_device_error() == 0
