"""Chunk-attention calls whose keys are cut into chunks (fa_extend_plan.cuh):
their inputs, made on the GPU, and attention over them in 64 bits. Run as a
script it writes the results of the library selected by FA_DEBUG_LIBRARY to the
file named on the command line."""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "tests")):
    if path not in sys.path:
        sys.path.insert(0, path)

BF, I32 = torch.bfloat16, torch.int32
TILE, PIECE, CTAS, ITEMS, L2 = 128, 320, 152, 6, 40 << 20

CASES = {  # kind, H, Hkv, d, block size, new tokens, cached tokens, chunks of each request's keys
    "boxes": ("bf16", 256, 4, 128, 16, [60], [60000], [3]),
    "boxes, two chunks": ("bf16", 16, 4, 128, 32, [1500], [40000], [2]),
    "boxes, five chunks": ("bf16", 256, 4, 128, 8, [36], [100000], [5]),
    "two requests": ("bf16", 96, 3, 64, 128, [160, 3, 80], [250000, 500, 170000], [2, 1, 2]),
    "gathered": ("bf16", 384, 3, 64, 3, [46], [200000], [3]),
    "gathered, others before and after": ("bf16", 256, 2, 128, 200, [1, 52, 2], [900, 230000, 2], [1, 3, 1]),
    "codes": ("q4", 256, 4, 128, 16, [66], [220000], [3]),
    "codes, two requests": ("q4", 96, 3, 64, 5, [160, 3, 130], [600000, 500, 500000], [2, 1, 2]),
}


def chunks(kind, H, Hkv, d, bs, new, lens, causal, max_blocks):
    """Into how many chunks each request's keys are cut, from the rule in words:
    no shorter than what fits L2 (all K/V heads' keys and values, 40 MB) and than
    a CTA's share of all items' keys, for requests of six items a head or more,
    and only where the context is 4.5 shares long at most (512 bytes a key and
    value: bf16, d = 128) or 2.5 (others)."""
    G = H // Hkv
    parts = -(-G // 128)
    tokens = 128 // -(-G // parts)          # a query tile's
    T, hv, span, ctx = sum(new), Hkv * parts, 2 * tokens, max_blocks * bs
    row = d // 2 + d // 16 if kind == "q4" else 2 * d
    lc = max(8 * TILE, L2 // (2 * Hkv * row) // TILE * TILE)
    items = hv * (T // span + min(T, len(new)))
    ctas = max(1, min(CTAS, items * (ctx + PIECE) // (5 * TILE)))
    if T <= (ITEMS - 1) * span or ctx <= lc:
        return [1] * len(new)
    keys = 0
    for n, length in zip(new, lens):
        for i in range(-(-n // span)):
            keys += hv * (max(0, length - n + min((i + 1) * span, n)) if causal else length)
    most = 4.5 if row == 256 else 2.5
    share = (keys // ctas + TILE) // TILE * TILE
    lc = max(lc, share)
    return [-(-length // lc) if -(-n // span) >= ITEMS and lc < length <= most * share else 1 for n, length in zip(new, lens)]


def inputs(name, seed, counting=False):
    """q, caches, table, lens, starts of a case, all on the GPU. counting: q is 0
    and dimension c of a value is 1 where its key tile's number is c modulo d,
    else 0, so o counts the keys that a token sees."""
    kind, H, Hkv, d, bs, new, lens, _ = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    nb = [-(-n // bs) for n in lens]
    total = sum(nb) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(I32)
    table = torch.zeros((len(new), max(nb)), dtype=I32, device="cuda")
    tile = torch.zeros((total, bs), dtype=torch.int64, device="cuda")  # the key tile of each slot
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = order[at:at + n]
        tile[table[b, :n].long()] = (torch.arange(n * bs, device="cuda") // TILE).view(n, bs)
        at += n
    q = torch.zeros((sum(new), H, d), dtype=BF, device="cuda") if counting else (4 * rn(sum(new), H, d)).to(BF)
    hit = (tile[:, None, :, None] % d == torch.arange(d, device="cuda")).expand(total, Hkv, bs, d)
    caches = []
    for n in "kv":
        if kind == "bf16":
            caches.append(hit.to(BF).contiguous() if counting and n == "v" else rn(total, Hkv, bs, d).to(BF))
            continue
        code = torch.randint(0, 16, (total, Hkv, bs, d), generator=g, device="cuda", dtype=torch.uint8)
        # steps and centres such that z + s (n - 8) is exact in fp32
        pair = torch.stack([0.1 + 0.3 * torch.rand((total, Hkv, bs, d // 64), generator=g, device="cuda"),
                            (0.3 * rn(total, Hkv, bs, d // 64) * 4096).round() / 4096], -1)
        if counting and n == "v":
            code, pair = 8 + hit.to(torch.uint8), torch.zeros_like(pair)
            pair[..., 0] = 1
        caches += [code[..., 0::2] | (code[..., 1::2] << 4), pair.to(BF)]
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    return q, caches, table, i32(lens), i32([sum(new[:b]) for b in range(len(new) + 1)])


def run(fa, q, caches, table, lens, starts, **kw):
    entry = fa.extend_paged if len(caches) == 2 else fa.extend_paged_q4
    return entry(q, *caches, table, lens, starts, **kw)


def held(caches, which, blocks, length):
    """[Hkv, length, d] of a request's keys (0) or values (1), in 64 bits."""
    flat = lambda t: t[blocks.long()].transpose(0, 1).flatten(1, 2)[:, :length]  # noqa: E731
    if len(caches) == 2:
        return flat(caches[which]).double()
    bytes_, pair = flat(caches[2 * which]), flat(caches[2 * which + 1]).float()
    code = torch.stack([bytes_ & 15, bytes_ >> 4], -1).flatten(-2).float() - 8
    x = pair[..., 1, None] + pair[..., 0, None] * code.unflatten(-1, (-1, 64))  # exact
    return x.flatten(-2).to(BF).double()


def attention64(q, caches, table, lens, starts, causal):
    """o, lse, Σ p |v| and max |k| Σ |q| scale of every row, in 64 bits."""
    T, H, d = q.shape
    Hkv, bs = caches[0].shape[1:3]
    o, around = (torch.zeros((T, H, d), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, reach = (torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, length in enumerate(lens.tolist()):
        lo, hi = starts[b].item(), starts[b + 1].item()
        if hi == lo or length == 0:
            continue
        blocks = table[b, :-(-length // bs)]
        K, V = held(caches, 0, blocks, length), held(caches, 1, blocks, length)
        sight = length - (hi - lo) + torch.arange(hi - lo, device="cuda")
        hidden = torch.arange(length, device="cuda") > sight[:, None]
        for h in range(H):
            k, v = K[h // (H // Hkv)], V[h // (H // Hkv)]
            Q = q[lo:hi, h].double()
            x = Q @ k.t() * d ** -0.5
            if causal:
                x.masked_fill_(hidden, -math.inf)
            lse[lo:hi, h] = torch.logsumexp(x, 1)
            p = x.sub_(lse[lo:hi, h, None]).exp_()
            o[lo:hi, h], around[lo:hi, h] = p @ v, p @ v.abs()
            reach[lo:hi, h] = k.abs().max() * Q.abs().sum(-1) * d ** -0.5
    return o, lse, around, reach


def main(path):
    import exact_tiled_attention_24_gb300 as fa
    assert fa.debug_checks() == (os.environ.get("FA_DEBUG_LIBRARY") == "1")
    out = {}
    for name in CASES:
        for causal in (True, False):
            o, lse = run(fa, *inputs(name, 7), causal=causal)
            torch.cuda.synchronize()
            assert fa.last_device_error() == 0
            out[f"{name} {causal} o"], out[f"{name} {causal} lse"] = o.cpu(), lse.cpu()
    torch.save(out, path)


if __name__ == "__main__":
    main(sys.argv[1])
