"""fp64 definitions of what stands between the projections and attention:
per-head norms, the position rotation, appends to a paged cache and the
4-bit codes a cache may be held in."""
import numpy as np

GROUP = 64  # dimensions that share one (step, centre) pair


def pair_indices(rot, interleaved):
    """Dimensions (first, second) of each rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rms(x, eps):
    """sqrt(mean_c x_c² + eps) over the last dimension, kept."""
    return np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def rotate(x, cos, sin, interleaved, sign=1.0):
    """Turn the pairs of x [..., d]; cos, sin [..., rot/2] broadcast against
    x's leading dimensions. sign = -1 turns back."""
    a, b = pair_indices(2 * cos.shape[-1], interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * cos - sign * x[..., b] * sin
    y[..., b] = x[..., b] * cos + sign * x[..., a] * sin
    return y


def _angles(cos, sin, positions, B, N):
    """The tables' rows of each token, [B, 1, N, rot/2]."""
    pos = np.broadcast_to(np.arange(N) if positions is None else np.asarray(positions), (B, N))
    return cos[pos][:, None], sin[pos][:, None]


def norm_rope(x, w=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """x [B, heads, N, d] -> the same shape; w None: no norm, cos None: no rotation."""
    if w is not None:
        x = x / rms(x, eps) * w
    if cos is None:
        return x.copy()
    return rotate(x, *_angles(cos, sin, positions, x.shape[0], x.shape[2]), interleaved)


def norm_rope_bwd(dy, x, w=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """dx and dw (None without a norm) for the output gradient dy."""
    g = dy if cos is None else rotate(dy, *_angles(cos, sin, positions, dy.shape[0], dy.shape[2]), interleaved, -1.0)
    if w is None:
        return g.copy(), None
    r = rms(x, eps)
    n = x / r
    h = g * w
    dx = (h - n * np.mean(h * n, axis=-1, keepdims=True)) / r
    return dx, (g * n).sum(axis=(0, 1, 2))


def bf16(x):
    """Nearest bf16 values (ties to even) of fp32 x, as fp32."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def q4_encode(x):
    """fp32 [..., d] -> codes [..., d] in 0..15, pairs [..., d/64, 2] (step,
    centre) as fp32 holding bf16 values: each operation in fp32, rounded by
    itself."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, GROUP)
    f = np.float32
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # NaN if any is
        half = f(0.5) * hi - f(0.5) * lo
        s = bf16(half * (f(1) / f(7.5)))
        z = bf16(f(0.5) * lo + f(0.5) * hi + f(0.5) * s)
        bad = ~(half < np.inf) | ~(np.abs(z) < np.inf)
        s, z = np.where(bad, f(np.nan), s), np.where(bad, f(np.nan), z)
        n = np.rint((g - z[..., None]) / np.where(s > 0, s, f(1))[..., None])
        n = np.where((s > 0)[..., None], np.clip(n, -8, 7), 0)
    return (n + 8).astype(np.uint8).reshape(x.shape), np.stack([s, z], -1)


def q4_pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def q4_unpack(packed):
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=np.int64)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def q4_values(codes, pairs):
    """The values held, in 64 bits."""
    n = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float64) - 8
    p = pairs.astype(np.float64)
    return (p[..., 1:] + p[..., :1] * n).reshape(codes.shape)


def append_slots(block_table, positions, requests, block_size):
    """(token, block, slot) of every token that is not padding."""
    out = []
    for t, pos in enumerate(positions):
        r = t if requests is None else int(requests[t])
        if r >= 0 and pos >= 0:
            out.append((t, int(block_table[r, pos // block_size]), int(pos) % block_size))
    return out


def extend_paged(q, k_cache, v_cache, block_table, seq_lens, q_starts, scale, causal=True):
    """q [T, H, d] -> o [T, H, d], lse [T, H] and Σ_j p_j |v_j| [T, H, d] (what
    a rounding of the weights acts on). Request b's tokens are rows q_starts[b]
    .. q_starts[b+1] - 1, the last of its seq_lens[b] cached tokens; rows of no
    request are zeros with lse = -inf."""
    T, H, d = q.shape
    Hkv, bs = k_cache.shape[1:3]
    o, around = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse = np.full((T, H), -np.inf)
    for b, L in enumerate(int(n) for n in seq_lens):
        lo, hi = int(q_starts[b]), int(q_starts[b + 1])
        t = np.arange(L)
        blocks = np.asarray(block_table)[b][t // bs]
        K, V = (c[blocks, :, t % bs] for c in (k_cache, v_cache))  # [L, Hkv, d]
        sight = L - (hi - lo) + np.arange(hi - lo) if causal else np.full(hi - lo, L - 1)
        for h in range(H):
            x = scale * (q[lo:hi, h] @ K[:, h // (H // Hkv)].T)
            x = np.where(t[None, :] <= sight[:, None], x, -np.inf)
            some = sight >= 0
            if L == 0 or not some.any():
                continue
            m = x[some].max(-1, keepdims=True)
            p = np.exp(x[some] - m)
            total = p.sum(-1, keepdims=True)
            rows = np.arange(lo, hi)[some]
            o[rows, h] = p @ V[:, h // (H // Hkv)] / total
            around[rows, h] = p @ np.abs(V[:, h // (H // Hkv)]) / total
            lse[rows, h] = (m + np.log(total))[:, 0]
    return o, lse, around
