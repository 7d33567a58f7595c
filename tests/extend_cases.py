"""Inputs of the chunk-attention tests: packed queries and a paged cache whose
blocks are placed at random, and the bounds that a result is held to."""
import numpy as np
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import extend_paged

BF = torch.bfloat16


def extend_case(H, Hkv, d, bs, new, lens, seed, before=0, after=0, q_std=1.0, fill=float("nan"), spare=3):
    """q [before + Σ new + after, H, d], caches, table, lengths and starts.
    Slots without a token hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    nb = [(n + bs - 1) // bs for n in lens]
    total = sum(nb) + spare
    T = before + sum(new) + after
    q = (torch.randn((T, H, d), generator=g) * q_std).to(BF)
    perm = torch.randperm(total, generator=g)
    table = torch.zeros((B, max(max(nb), 1)), dtype=torch.int32)
    used = torch.zeros((total, bs), dtype=torch.bool)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]].to(torch.int32)
        t = torch.arange(lens[b])
        used[perm[at:at + nb[b]][t // bs], t % bs] = True
        at += nb[b]
    caches = []
    for _ in "kv":
        c = torch.randn((total, Hkv, bs, d), generator=g).to(BF)
        c[~used[:, None, :].expand(total, Hkv, bs)] = fill
        caches.append(c)
    starts = torch.tensor([before] + new).cumsum(0).to(torch.int32)
    return q, caches, table, torch.tensor(lens, dtype=torch.int32), starts


def run(fa, q, caches, table, lens, starts, **kw):
    entry = fa.extend_paged if len(caches) == 2 else fa.extend_paged_q4
    o, lse = entry(q.cuda(), *(c.cuda() for c in caches), table.cuda(), lens.cuda(), starts.cuda(), **kw)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    return o, lse


def check(q, K, V, table, lens, starts, o, lse, causal=True, scale=None):
    """Bounds. Each weight is rounded to bf16 before the product with V (half a
    step, 2^-8): at most 2^-8 Σ p |v|; the result once: 2^-8 |o|. A score is an
    fp32 sum of d <= 128 products, under 2^7 roundings of 2^-24 of Σ|q k| (twice
    that where the tensor core truncates), so off by at most e = 2^-16 max|k|
    Σ|q| · scale in natural units; weights by 2 e relatively, o by 2 e Σ p |v|,
    lse by e plus the logarithm's and the sum's 2^-20 (|lse| + 1). The factor
    1.01 covers fp32 sums and exponentials (2^-20 of Σ p |v| together)."""
    Q, K, V = to_f64(q), np.nan_to_num(K), np.nan_to_num(V)
    d = Q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    ro, rl, around = extend_paged(Q, K, V, table.numpy(), lens.numpy(), starts.numpy(), scale, causal)
    e = 2.0 ** -16 * np.abs(K).max() * np.abs(Q).sum(-1) * scale
    tol = (2.0 ** -8 * (around + np.abs(ro)) + 2 * e[..., None] * around) * 1.01
    err = np.abs(to_f64(o) - ro)
    assert np.all(err <= tol), f"o: {(err - tol).max()} over, at {np.unravel_index((err - tol).argmax(), err.shape)}"
    got = lse.double().cpu().numpy()
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(got), none)
    dl = np.abs(got[~none] - rl[~none])
    assert np.all(dl <= e[~none] + 2.0 ** -20 * (np.abs(rl[~none]) + 1)), f"lse: {dl.max()}"
