"""The operators between a layer's projections and attention over a cache,
as cases that can be measured: per-head norms with the position rotation
(training, forward and backward), appending to a paged cache in bf16 or in
4 bits, and one decode step's attention over a 4-bit cache.

`run` computes a case in plain torch operations (`own` false) or through the
package's entry points (`own` true). `exact` computes it in 64 bits from the
definition.

A 4-bit cache holds, for each token and K/V head, d codes n in 0..15 (two a
byte, the even dimension in the low half) and, for each group of 64
dimensions, a bf16 pair (s, z): the value held is z + s (n - 8).
"""
import math

import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # A training step's q and k, views of a packed projection, 8 K/V heads.
        {"name": "norm_rope train fwd", "op": "norm_rope", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128, "rot": 128,
         "norm": True, "interleaved": False, "packed": True, "documents": False},
        # The same step's backward: gradients of q, k and both weights.
        {"name": "norm_rope train bwd", "op": "norm_rope_bwd", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128,
         "rot": 128, "norm": True, "interleaved": False, "packed": True, "documents": False},
        # Small heads, an odd length, half of each head rotated, several documents in a row.
        {"name": "norm_rope ragged fwd", "op": "norm_rope", "B": 4, "H": 12, "Hkv": 12, "N": 1028, "d": 64, "rot": 32,
         "norm": True, "interleaved": True, "packed": False, "documents": True},
        {"name": "norm_rope ragged bwd", "op": "norm_rope_bwd", "B": 4, "H": 12, "Hkv": 12, "N": 1028, "d": 64,
         "rot": 32, "norm": True, "interleaved": True, "packed": False, "documents": True},
        # One new token for each of 32 requests, 2k to 8k tokens into their contexts.
        {"name": "append step", "op": "append", "T": 32, "requests": 32, "pad": 0, "H": 32, "Hkv": 8, "d": 128,
         "rot": 128, "norm": True, "interleaved": False, "bs": 16, "at": 2048, "q4": False},
        # Prompts of different lengths in one batch, padded at its end.
        {"name": "append prompts", "op": "append", "T": 16384, "requests": 7, "pad": 100, "H": 32, "Hkv": 8, "d": 128,
         "rot": 128, "norm": True, "interleaved": False, "bs": 16, "at": 0, "q4": False},
        {"name": "append q4 step", "op": "append", "T": 32, "requests": 32, "pad": 0, "H": 32, "Hkv": 8, "d": 128,
         "rot": 128, "norm": False, "interleaved": False, "bs": 16, "at": 2048, "q4": True},
        {"name": "append q4 prompts", "op": "append", "T": 16384, "requests": 7, "pad": 100, "H": 32, "Hkv": 8,
         "d": 128, "rot": 128, "norm": False, "interleaved": False, "bs": 16, "at": 0, "q4": True},
        # 32 requests with 2k to 8k cached tokens each.
        {"name": "decode q4 batch", "op": "decode", "B": 32, "H": 32, "Hkv": 8, "d": 128, "bs": 16, "shortest": 2048,
         "longest": 8192},
        # Two long contexts: the work of few requests has to be spread.
        {"name": "decode q4 long", "op": "decode", "B": 2, "H": 32, "Hkv": 8, "d": 128, "bs": 64, "shortest": 100000,
         "longest": 131072},
        # A handful of short requests, one of them empty: latency.
        {"name": "decode q4 short", "op": "decode", "B": 3, "H": 12, "Hkv": 12, "d": 64, "bs": 16, "shortest": 0,
         "longest": 700},
        # One token a cache block, 16 query heads for a K/V head.
        {"name": "decode q4 one-token blocks", "op": "decode", "B": 16, "H": 32, "Hkv": 2, "d": 128, "bs": 1,
         "shortest": 1000, "longest": 8192},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "append", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    H = Hkv * rng.choice([1, 2, 4, 5, 8] if Hkv > 2 else [1, 2, 4, 7, 8, 16])
    if op == "decode":
        longest = _log_int(rng, 1, 131072)
        most = max(1, min(48, 1_000_000 // (longest * Hkv)))
        return {"op": op, "B": _log_int(rng, 1, most), "H": H, "Hkv": Hkv, "d": d,
                "bs": rng.choice([1, 3, 8, 16, 16, 32, 48, 64, 128]), "shortest": rng.randint(0, longest),
                "longest": longest}
    rot = rng.choice([d, d, d // 2, 16, 48])
    both = {"H": H, "Hkv": Hkv, "d": d, "rot": rot, "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.3}
    if op == "append":
        T = _log_int(rng, 1, max(1, 786432 // (H + 2 * Hkv)) if H + 2 * Hkv > 48 else 16384)
        return {"op": op, "T": T, "requests": rng.randint(1, min(T, 64)), "pad": rng.randint(0, 9),
                "bs": rng.choice([1, 5, 8, 16, 32, 64]), "at": rng.choice([0, rng.randint(1, 30000)]),
                "q4": rng.random() < 0.5, **both}
    B = rng.randint(1, 4)
    N = _log_int(rng, 1, min(16384, 655360 // (B * (H + Hkv))))
    return {"op": op, "B": B, "N": N, "packed": rng.random() < 0.5, "documents": rng.random() < 0.3, **both}


def work(case):
    c = case
    if c["op"] == "decode":
        tokens = sum(_lengths(c))
        return {"bytes": 2 * tokens * c["Hkv"] * (c["d"] // 2 + c["d"] // 16)
                + c["B"] * c["H"] * (4 * c["d"] + 4),
                "flops": 4 * tokens * c["H"] * c["d"]}
    tables = 4 * c["rot"]  # one position's cosines and sines
    if c["op"] == "append":
        row = 2 * c["d"]
        kv = 2 * c["Hkv"] * (c["d"] // 2 + c["d"] // 16 + row if c["q4"] else row)
        return {"bytes": c["T"] * (2 * c["H"] * row + 2 * c["Hkv"] * row + kv + 8 + tables), "flops": 0}
    rows = c["B"] * c["N"] * (c["H"] + c["Hkv"])
    passes = 2 if c["op"] == "norm_rope" or not c["norm"] else 3
    return {"bytes": passes * rows * c["d"] * 2 + c["N"] * tables, "flops": 0}


def _lengths(c):
    """Cached tokens of a decode case's requests, from its own numbers."""
    B, lo, hi = c["B"], c["shortest"], c["longest"]
    return [hi - (hi - lo) * ((7 * b) % B) // max(1, B - 1) for b in range(B)]


# ------------------------------------------------------------------- inputs

def _tables(positions, rot):
    """Cosines and sines of positions 0 .. positions-1, angles in 64 bits."""
    inverse = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angles = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inverse
    return angles.cos().float(), angles.sin().float()


def _weights(c, g):
    if not c["norm"]:
        return None, None
    draw_one = lambda: (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(BF16)  # noqa: E731
    return draw_one(), draw_one()


def _keys(x, g):
    """Keys have a few channels far larger than the others."""
    large = torch.rand(x.shape[-1], generator=g, device="cuda") < 0.05
    return x * torch.where(large, 4.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    c = dict(case)
    if c["op"] == "decode":
        return {"case": c, **_prepare_decode(c, g)}
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    qw, kw = _weights(c, g)
    if c["op"] == "append":
        T, R, bs = c["T"], c["requests"], c["bs"]
        qkv = randn(T + c["pad"], H + 2 * Hkv, d)
        qkv[:, H:H + Hkv] = _keys(qkv[:, H:H + Hkv], g)
        qkv = qkv.to(BF16)
        share, rest = divmod(T, R)  # the first request has the rest too
        first = torch.randint(0, c["at"] + 1, (R,), generator=g, device="cuda") + c["at"]
        token = torch.arange(T, device="cuda")
        request = ((token - rest).clamp(min=0) // share)
        start = torch.where(request > 0, request * share + rest, 0)
        position = first[request] + token - start
        pad = torch.full((c["pad"],), -1, device="cuda", dtype=torch.int64)
        longest = 2 * c["at"] + share + rest + 1
        blocks = -(-longest // bs)
        spare = 5
        # a request's earlier blocks are not touched here: all of them share block 0
        fresh = -(-(share + rest) // bs) + 1
        total = 1 + R * fresh + spare
        order = torch.randperm(total - 1, generator=g, device="cuda")[:R * fresh].view(R, fresh) + 1
        at = torch.arange(blocks, device="cuda")[None, :] - (first // bs)[:, None]
        inside = (at >= 0) & (at < fresh)
        table = torch.where(inside, order.gather(1, at.clamp(0, fresh - 1)), 0).to(torch.int32)
        s = {"case": c, "q": qkv[:, :H], "k": qkv[:, H:H + Hkv], "v": qkv[:, H + Hkv:], "table": table,
             "positions": torch.cat([position, pad]).to(torch.int32), "requests": torch.cat([request, pad]).to(torch.int32),
             "q_weight": qw, "k_weight": kw, "q_out": torch.zeros((T + c["pad"], H, d), dtype=BF16, device="cuda")}
        s["cos"], s["sin"] = _tables(longest, c["rot"])
        if c["q4"]:
            for n in "kv":
                s[n + "_cache"] = torch.zeros((total, Hkv, bs, d // 2), dtype=torch.uint8, device="cuda")
                s[n + "_scale"] = torch.zeros((total, Hkv, bs, d // 64, 2), dtype=BF16, device="cuda")
                s[n + "_values"] = torch.zeros((T + c["pad"], Hkv, d), dtype=BF16, device="cuda")
        else:
            for n in "kv":
                s[n + "_cache"] = torch.zeros((total, Hkv, bs, d), dtype=BF16, device="cuda")
        return s
    B, N = c["B"], c["N"]
    if c["packed"]:  # the projection's output, one token's heads side by side
        qkv = randn(B, N, H + 2 * Hkv, d).to(BF16)
        q, k = (x.transpose(1, 2) for x in (qkv[:, :, :H], qkv[:, :, H:H + Hkv]))
    else:
        q, k = randn(B, H, N, d).to(BF16), randn(B, Hkv, N, d).to(BF16)
    positions = None
    if c["documents"]:  # positions start again at each document
        starts = torch.rand((B, N), generator=g, device="cuda") < 4.0 / N
        index = torch.arange(N, device="cuda").expand(B, N)
        positions = (index - torch.where(starts, index, 0).cummax(1).values).to(torch.int32)
    s = {"case": c, "q": q, "k": k, "positions": positions, "q_weight": qw, "k_weight": kw}
    s["cos"], s["sin"] = _tables(N, c["rot"])
    if c["op"] == "norm_rope_bwd":
        s["dq_out"], s["dk_out"] = randn(B, H, N, d).to(BF16), randn(B, Hkv, N, d).to(BF16)
    return s


def _prepare_decode(c, g):
    B, H, Hkv, d, bs = c["B"], c["H"], c["Hkv"], c["d"], c["bs"]
    lens = torch.tensor(_lengths(c), device="cuda")
    count = -(-lens // bs)
    width = max(1, int(-(-c["longest"] // bs)))
    total = sum(-(-n // bs) for n in _lengths(c)) + 3
    order = torch.randperm(total, generator=g, device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    before = (count.cumsum(0) - count)[:, None]
    table = torch.where(slot < count[:, None], order[(before + slot).clamp(max=total - 1)], 0).to(torch.int32)
    used = torch.zeros((total, bs), dtype=torch.bool, device="cuda")
    token = torch.arange(width * bs, device="cuda")[None, :].expand(B, -1)
    live = token < lens[:, None]
    used[table.long().gather(1, token // bs)[live], (token % bs)[live]] = True
    s = {"q": torch.randn((B, H, d), generator=g, device="cuda").to(BF16), "table": table, "lens": lens.to(torch.int32)}
    for n in "kv":
        code = (torch.randn((total, Hkv, bs, d), generator=g, device="cuda") * 3 + 8).round().clamp(0, 15).to(torch.uint8)
        s[n + "_cache"] = code[..., 0::2] | (code[..., 1::2] << 4)
        pair = torch.stack([0.25 + 0.15 * torch.rand((total, Hkv, bs, d // 64), generator=g, device="cuda"),
                            0.15 * torch.randn((total, Hkv, bs, d // 64), generator=g, device="cuda")], -1)
        # slots that hold no token hold whatever was there
        s[n + "_scale"] = torch.where(used[:, None, :, None, None], pair, float("nan")).to(BF16)
    return s


# --------------------------------------------------------------- plain forms

def _norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)


def _pairs(x, rot, interleaved):
    """The two members of each rotated pair."""
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, interleaved):
    both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _rotate(x, cos, sin, rot, interleaved):
    a, b = _pairs(x, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, x[..., rot:], interleaved)


def _prepared(x, w, cos, sin, c):
    return _rotate(_norm(x, w), cos, sin, c["rot"], c["interleaved"])


def _plain_norm_rope(s):
    c = s["case"]
    cos, sin = _at(s, s["cos"], s["sin"])
    return {"q": _prepared(s["q"].float(), s["q_weight"], cos, sin, c).to(BF16),
            "k": _prepared(s["k"].float(), s["k_weight"], cos, sin, c).to(BF16)}


def _at(s, cos, sin):
    """The tables' rows of each token, to go with [B, heads, N, d]."""
    if s["positions"] is None:
        return cos[:s["case"]["N"]], sin[:s["case"]["N"]]
    rows = s["positions"].long()
    return cos[rows][:, None], sin[rows][:, None]


def _back(dy, x, w, cos, sin, c):
    """Gradients of the norm and rotation of x: dx, dw."""
    g = _rotate(dy, cos, -sin, c["rot"], c["interleaved"])
    if w is None:
        return g, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = g * w.to(x.dtype)
    dw = (g * (x * r)).sum((0, 1, 2), dtype=torch.float64)
    return r * (h - x * (r * r * (h * x).mean(-1, keepdim=True))), dw


def _plain_norm_rope_bwd(s):
    c = s["case"]
    cos, sin = _at(s, s["cos"], s["sin"])
    dq, dqw = _back(s["dq_out"].float(), s["q"].float(), s["q_weight"], cos, sin, c)
    dk, dkw = _back(s["dk_out"].float(), s["k"].float(), s["k_weight"], cos, sin, c)
    out = {"dq": dq.to(BF16), "dk": dk.to(BF16)}
    return out if dqw is None else {**out, "dq_weight": dqw.float(), "dk_weight": dkw.float()}


def _quantise(x):
    """[..., d] -> codes 0..15 [..., d], (s, z) [..., d/64, 2] in bf16."""
    grouped = x.unflatten(-1, (-1, 64))
    low, high = grouped.amin(-1), grouped.amax(-1)
    step = ((0.5 * high - 0.5 * low) * (1 / 7.5)).to(BF16).to(x.dtype)
    centre = (0.5 * low + 0.5 * high + 0.5 * step).to(BF16).to(x.dtype)
    # a division, not a product with 1 / step: bf16 values often lie exactly between two codes
    code = ((grouped - centre[..., None]) / torch.where(step > 0, step, math.inf)[..., None]).round().add(8).clamp(0, 15)
    return code.flatten(-2), torch.stack([step, centre], -1)


def _held(code, pair):
    """The values that codes and pairs stand for."""
    return (pair[..., 1, None] + pair[..., 0, None] * (code.unflatten(-1, (-1, 64)) - 8)).flatten(-2)


def _plain_append(s):
    c = s["case"]
    n, bs = c["T"], c["bs"]
    position, request = s["positions"][:n].long(), s["requests"][:n].long()
    cos, sin = s["cos"][position][:, None], s["sin"][position][:, None]
    block, slot = s["table"][request, position // bs].long(), position % bs
    s["q_out"][:n] = _prepared(s["q"][:n].float(), s["q_weight"], cos, sin, c).to(BF16)
    new = (("k", _prepared(s["k"][:n].float(), s["k_weight"], cos, sin, c)), ("v", s["v"][:n].float()))
    if not c["q4"]:
        for name, x in new:
            s[name + "_cache"][block, :, slot] = x.to(BF16)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    for name, x in new:
        code, pair = _quantise(x)
        s[name + "_values"][:n] = _held(code, pair).to(BF16)
        byte = code.to(torch.uint8)
        s[name + "_cache"][block, :, slot] = byte[..., 0::2] | (byte[..., 1::2] << 4)
        s[name + "_scale"][block, :, slot] = pair.to(BF16)
    return {"q": s["q_out"], "k_values": s["k_values"], "v_values": s["v_values"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _gathered(cache, scale, table, bs, length):
    """[B, Hkv, length, d] values of the first `length` tokens of each request."""
    token = torch.arange(length, device="cuda")
    block, slot = table[:, token // bs].long(), token % bs
    byte = cache[block, :, slot]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).float()
    return _held(code, scale[block, :, slot].float()).transpose(1, 2)


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, d, longest = c["B"], c["H"], c["Hkv"], c["d"], c["longest"]
    lens = s["lens"]
    if longest == 0:
        return {"o": torch.zeros_like(s["q"]), "lse": torch.full((B, H), -math.inf, device="cuda")}
    dead = (torch.arange(longest, device="cuda")[None, :] >= lens[:, None])[:, None, :, None]
    keys = _gathered(s["k_cache"], s["k_scale"], s["table"], c["bs"], longest).masked_fill(dead, 0.0)
    values = _gathered(s["v_cache"], s["v_scale"], s["table"], c["bs"], longest).masked_fill(dead, 0.0)
    q = s["q"].float().view(B, Hkv, H // Hkv, d)
    scores = (torch.matmul(q, keys.transpose(2, 3)) * d ** -0.5).masked_fill(dead.transpose(2, 3), -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(total > 0, total, 1.0)
    return {"o": o.reshape(B, H, d).to(BF16), "lse": (top + total.log()).reshape(B, H)}


# ---------------------------------------------------------------------- runs

def _own_run(s):
    import exact_tiled_attention_24_gb300 as fa
    c = s["case"]
    if c["op"] == "norm_rope":
        q, k = fa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return {"q": q, "k": k}
    if c["op"] == "norm_rope_bwd":
        dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["cos"], s["sin"],
                                               positions=s["positions"], q_weight=s["q_weight"],
                                               k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        return {"dq": dq, "dk": dk} if dqw is None else {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if c["op"] == "decode":
        o, lse = fa.decode_paged_q4(s["q"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"], s["table"],
                                    s["lens"], n_splits=0)
        return {"o": o, "lse": lse}
    common = dict(requests=s["requests"], cos=s["cos"], sin=s["sin"], q=s["q"], q_weight=s["q_weight"],
                  k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"], q_out=s["q_out"])
    if not c["q4"]:
        fa.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["positions"], **common)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    fa.append_paged_q4(s["k"], s["v"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"], s["table"],
                       s["positions"], k_values=s["k_values"], v_values=s["v_values"], **common)
    return {"q": s["q_out"], "k_values": s["k_values"], "v_values": s["v_values"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm_rope":
        return _plain_norm_rope(state)
    if op == "norm_rope_bwd":
        return _plain_norm_rope_bwd(state)
    if op == "append":
        return _plain_append(state)
    return _plain_decode(state)


# ------------------------------------------------------------- in 64 bits

def _exact_turned(x, w, angle_rows, c, sign=1.0):
    """Norm (w given), then each pair as a complex number times e^(i angle).
    angle_rows = (cos, sin) in 64 bits, broadcast against x's pairs."""
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    rot = c["rot"]
    order = torch.arange(rot, device="cuda")
    order = order.view(-1, 2) if c["interleaved"] else order.view(2, -1).t()
    turn = torch.complex(*angle_rows)
    z = torch.view_as_complex(x[..., order].contiguous()) * (turn if sign > 0 else turn.conj())
    y = x.clone()
    y[..., order] = torch.view_as_real(z)
    return y


def _exact_append(s):
    c, n, bs = s["case"], s["case"]["T"], s["case"]["bs"]
    position, request = s["positions"][:n].long(), s["requests"][:n].long()
    turn = (s["cos"].double()[position][:, None], s["sin"].double()[position][:, None])
    block = s["table"].long()[request, torch.div(position, bs, rounding_mode="floor")]
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q[:n] = _exact_turned(s["q"][:n].double(), s["q_weight"], turn, c)
    out = {"q": q}
    for name, x in (("k", _exact_turned(s["k"][:n].double(), s["k_weight"], turn, c)), ("v", s["v"][:n].double())):
        if not c["q4"]:
            cache = s[name + "_cache"].double()
            cache[block, :, position % bs] = x
            out[name + "_cache"] = cache
            continue
        g = x.reshape(*x.shape[:-1], -1, 64)
        low, high = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        step = ((high - low) / 15).to(BF16).double()
        centre = ((low + high + step) / 2).to(BF16).double()
        level = torch.where(step > 0, (g - centre) / step, torch.zeros_like(g)).round().clamp(-8, 7)
        values = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
        values[:n] = (centre + step * level).reshape(x.shape)
        scale = s[name + "_scale"].double()
        scale[block, :, position % bs] = torch.cat([step, centre], -1)
        out[name + "_values"], out[name + "_scale"] = values, scale
    return out


def _exact_decode(s):
    c = s["case"]
    H, Hkv, d, bs = c["H"], c["Hkv"], c["d"], c["bs"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(_lengths(c)):
        if length == 0:
            continue
        blocks = s["table"][b, :-(-length // bs)].long()
        held = []
        for name in "kv":
            byte = s[name + "_cache"][blocks].transpose(1, 2).reshape(-1, Hkv, d // 2)[:length].int()
            pair = s[name + "_scale"][blocks].transpose(1, 2).reshape(-1, Hkv, d // 64, 1, 2)[:length].double()
            code = torch.empty((length, Hkv, d), dtype=torch.float64, device="cuda")
            code[..., 0::2], code[..., 1::2] = (byte % 16).double(), torch.div(byte, 16, rounding_mode="floor").double()
            held.append((pair[..., 1] + pair[..., 0] * (code.view(length, Hkv, -1, 64) - 8)).reshape(length, Hkv, d))
        for h in range(H):
            head = h // (H // Hkv)
            x = held[0][:, head] @ s["q"][b, h].double() / math.sqrt(d)
            lse[b, h] = torch.logsumexp(x, 0)
            o[b, h] = torch.exp(x - lse[b, h]) @ held[1][:, head]
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "decode":
        return _exact_decode(s)
    rows = torch.arange(c["N"], device="cuda").expand(c["B"], -1) if s["positions"] is None else s["positions"].long()
    turn = (s["cos"].double()[rows][:, None], s["sin"].double()[rows][:, None])
    out = {}
    for name in "qk":
        x, w = s[name].double(), s[name + "_weight"]
        if c["op"] == "norm_rope":
            out[name] = _exact_turned(x, w, turn, c)
            continue
        g = _exact_turned(s["d" + name + "_out"].double(), None, turn, c, sign=-1.0)
        if w is not None:  # y = u w with u = x / |x|rms: du = g w, less its part along u
            rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            u = x / rms
            out["d" + name + "_weight"] = (g * u).sum((0, 1, 2))
            g = g * w.double()
            g = (g - u * (g * u).mean(-1, keepdim=True)) / rms
        out["d" + name] = g
    return out
