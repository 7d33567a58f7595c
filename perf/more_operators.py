"""Attention of chunks of new tokens over a paged cache (bf16 or 4-bit codes)
and position rotations with several axes, as cases that can be measured.

`run` computes a case in plain torch operations (`own` false) or through the
package's entry points (`own` true). `exact` computes it in 64 bits from the
definition.

A chunk: request b's new tokens are rows q_starts[b] .. q_starts[b + 1] - 1 of
q [T, H, d], and they are the last of its seq_lens[b] cached tokens; a token at
position p sees keys 0 .. p. A 4-bit cache holds, for each token and K/V head,
d codes n in 0..15 (two a byte, the even dimension in the low half) and, for
each group of 64 dimensions, a bf16 pair (s, z): chunks read the value
z + s (n - 8) rounded to bf16, which is what an append hands out as the value
held.

Several axes: pair i of the rotated dimensions turns by the angle of the
token's position on one axis (time, height or width), the pairs dealt to the
axes in sections.
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
        # A whole prompt of 8192 tokens, nothing cached before it.
        {"name": "extend prompt", "op": "extend", "q4": False, "B": 1, "H": 32, "Hkv": 8, "d": 128, "bs": 16,
         "new_least": 8192, "new_most": 8192, "shortest": 8192, "longest": 8192},
        # A serving step: prompts in chunks of different lengths beside requests that bring a few tokens.
        {"name": "extend chunks", "op": "extend", "q4": False, "B": 12, "H": 32, "Hkv": 8, "d": 128, "bs": 16,
         "new_least": 1, "new_most": 512, "shortest": 2048, "longest": 8192},
        # Five drafted tokens a request, to be verified: the cache's bytes are what it costs.
        {"name": "extend drafts", "op": "extend", "q4": False, "B": 32, "H": 32, "Hkv": 8, "d": 128, "bs": 16,
         "new_least": 5, "new_most": 5, "shortest": 2048, "longest": 8192},
        # The last chunk of a very long prompt.
        {"name": "extend long", "op": "extend", "q4": False, "B": 1, "H": 32, "Hkv": 8, "d": 128, "bs": 64,
         "new_least": 1024, "new_most": 1024, "shortest": 131072, "longest": 131072},
        # A handful of short requests, small heads, an odd block size: latency.
        {"name": "extend short", "op": "extend", "q4": False, "B": 3, "H": 12, "Hkv": 12, "d": 64, "bs": 5,
         "new_least": 1, "new_most": 37, "shortest": 40, "longest": 700},
        # The serving step, the drafts and a long prompt's chunk over a cache in 4 bits.
        {"name": "extend q4 chunks", "op": "extend", "q4": True, "B": 12, "H": 32, "Hkv": 8, "d": 128, "bs": 16,
         "new_least": 1, "new_most": 512, "shortest": 2048, "longest": 8192},
        {"name": "extend q4 drafts", "op": "extend", "q4": True, "B": 32, "H": 32, "Hkv": 8, "d": 128, "bs": 16,
         "new_least": 5, "new_most": 5, "shortest": 2048, "longest": 8192},
        {"name": "extend q4 long", "op": "extend", "q4": True, "B": 1, "H": 32, "Hkv": 8, "d": 128, "bs": 64,
         "new_least": 300, "new_most": 300, "shortest": 131072, "longest": 131072},
        # A training step's q and k of video tokens, views of a packed projection; forward and gradients.
        {"name": "axes train fwd", "op": "norm_rope", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128,
         "time": 16, "height": 24, "width": 24, "dealt": False, "norm": True, "interleaved": False},
        {"name": "axes train bwd", "op": "norm_rope_bwd", "B": 2, "H": 32, "Hkv": 8, "N": 8192, "d": 128,
         "time": 16, "height": 24, "width": 24, "dealt": False, "norm": True, "interleaved": False},
        # Prompts with images in them, into the cache; the axes dealt to the pairs in turn.
        {"name": "axes append prompts", "op": "append", "q4": False, "T": 16384, "requests": 7, "pad": 100, "H": 32,
         "Hkv": 8, "d": 128, "time": 24, "height": 20, "width": 20, "dealt": True, "norm": True, "interleaved": False,
         "bs": 16},
        # One new token for each of 32 requests into 4-bit codes, its rotary position behind its slot.
        {"name": "axes append q4 step", "op": "append", "q4": True, "T": 32, "requests": 32, "pad": 0, "H": 32,
         "Hkv": 8, "d": 128, "time": 16, "height": 24, "width": 24, "dealt": False, "norm": False, "interleaved": False,
         "bs": 16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "extend", "extend", "norm_rope", "norm_rope_bwd", "append"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    H = Hkv * rng.choice([1, 2, 4, 5, 8] if Hkv > 2 else [1, 2, 4, 7, 8, 16])
    if op == "extend":
        longest = _log_int(rng, 1, 131072)
        most = min(longest, 8192, max(1, int(2.0e12 / (512 * H * longest))))
        new_most = _log_int(rng, 1, most)
        # what fits: the plain form's scores of the whole batch, and the cache
        B = min(48, 4_000_000_000 // (H * new_most * longest), 1_500_000 // (longest * Hkv))
        return {"op": op, "q4": rng.random() < 0.4, "B": _log_int(rng, 1, max(1, B)), "H": H, "Hkv": Hkv, "d": d,
                "bs": rng.choice([1, 3, 8, 16, 16, 32, 48, 64, 128]), "new_least": rng.randint(0, new_most),
                "new_most": new_most, "shortest": rng.randint(new_most, longest), "longest": longest}
    pairs = rng.choice([d, d, d // 2, 48]) // 2
    first = rng.randint(1, pairs - 2)
    second = rng.randint(1, pairs - first - 1)
    both = {"H": H, "Hkv": Hkv, "d": d, "time": first, "height": second, "width": pairs - first - second,
            "dealt": rng.random() < 0.3, "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.3}
    if op == "append":
        T = _log_int(rng, 1, min(16384, 786432 // (H + 2 * Hkv)))
        return {"op": op, "q4": rng.random() < 0.5, "T": T, "requests": rng.randint(1, min(T, 64)),
                "pad": rng.randint(0, 9), "bs": rng.choice([1, 5, 8, 16, 32, 64]), **both}
    B = rng.randint(1, 4)
    return {"op": op, "B": B, "N": _log_int(rng, 1, min(16384, 655360 // (B * (H + Hkv)))), **both}


def _spread(lo, hi, B, stride):
    """B numbers from lo to hi, in no order (its own numbers: the case alone decides)."""
    return [hi - (hi - lo) * ((stride * b) % B) // max(1, B - 1) for b in range(B)]


def _lengths(c):
    """(cached tokens, new tokens) of an extend case's requests."""
    return _spread(c["shortest"], c["longest"], c["B"], 7), _spread(c["new_least"], c["new_most"], c["B"], 5)


def work(case):
    c = case
    if c["op"] == "extend":
        lens, new = _lengths(c)
        row = c["d"] // 2 + c["d"] // 16 if c["q4"] else 2 * c["d"]
        # a request that brings nothing has nothing read
        seen = sum(n for n, m in zip(lens, new) if m > 0)
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
        return {"bytes": 2 * seen * c["Hkv"] * row + sum(new) * c["H"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["H"] * pairs}
    rot = 2 * (c["time"] + c["height"] + c["width"])
    tables = 4 * rot + 12  # one token's cosines and sines, its three positions
    row = 2 * c["d"]
    if c["op"] == "append":
        kv = 2 * c["Hkv"] * (c["d"] // 2 + c["d"] // 16 + row if c["q4"] else row)
        return {"bytes": c["T"] * (2 * c["H"] * row + 2 * c["Hkv"] * row + kv + 8 + tables), "flops": 0}
    rows = c["B"] * c["N"] * (c["H"] + c["Hkv"])
    passes = 2 if c["op"] == "norm_rope" or not c["norm"] else 3
    return {"bytes": passes * rows * row + c["B"] * c["N"] * tables, "flops": 0}


# ------------------------------------------------------------------- inputs

def _tables(positions, rot):
    """Cosines and sines of positions 0 .. positions-1, angles in 64 bits."""
    inverse = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angles = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inverse
    return angles.cos().float(), angles.sin().float()


def _axis_of_pair(c):
    """The axis of each rotated pair: section after section, or dealt in turn while an axis has pairs left."""
    left = [c["time"], c["height"], c["width"]]
    if not c["dealt"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _weights(c, g):
    if not c["norm"]:
        return None, None
    draw_one = lambda: (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(BF16)  # noqa: E731
    return draw_one(), draw_one()


def _keys(x, g):
    """Keys have a few channels far larger than the others."""
    large = torch.rand(x.shape[-1], generator=g, device="cuda") < 0.05
    return x * torch.where(large, 4.0, 1.0)


def _grid_positions(n, g):
    """[3, n] int32: text, whose three positions are equal, with frames of a 20 x 28 grid from a random token on."""
    token = torch.arange(n, device="cuda")
    start = int(torch.randint(0, max(1, n // 4) + 1, (1,), generator=g, device="cuda"))
    at = (token - start).clamp(min=0)
    time, rest = at // 560, at % 560
    image = (token >= start) & (token < start + 560 * max(1, n // 1120))
    text = torch.where(token < start, token, torch.minimum(token, start + 28 + at // 560))
    p = torch.stack([torch.where(image, start + time, text), torch.where(image, start + rest // 28, text),
                     torch.where(image, start + rest % 28, text)])
    return p.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    c = dict(case)
    if c["op"] == "extend":
        return {"case": c, **_prepare_extend(c, g)}
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    qw, kw = _weights(c, g)
    pairs = _axis_of_pair(c)
    s = {"case": c, "axes": bytes(pairs), "axis_of_pair": torch.tensor(pairs, device="cuda"), "q_weight": qw,
         "k_weight": kw}
    rot = 2 * len(pairs)
    if c["op"] == "append":
        T, R, bs = c["T"], c["requests"], c["bs"]
        qkv = randn(T + c["pad"], H + 2 * Hkv, d)
        qkv[:, H:H + Hkv] = _keys(qkv[:, H:H + Hkv], g)
        qkv = qkv.to(BF16)
        share, rest = divmod(T, R)  # the first request has the rest too
        token = torch.arange(T, device="cuda")
        request = (token - rest).clamp(min=0) // share
        before = 11  # cached already
        position = before + token - torch.where(request > 0, request * share + rest, 0)
        pad = torch.full((c["pad"],), -1, device="cuda", dtype=torch.int64)
        longest = before + share + rest
        blocks = -(-longest // bs)
        order = torch.randperm(R * blocks + 3, generator=g, device="cuda")[:R * blocks]
        rope = _grid_positions(T + c["pad"], g)
        rope[:, T:] = -1  # padding has no positions
        s |= {"q": qkv[:, :H], "k": qkv[:, H:H + Hkv], "v": qkv[:, H + Hkv:], "table": order.view(R, blocks).to(torch.int32),
              "positions": torch.cat([position, pad]).to(torch.int32), "requests": torch.cat([request, pad]).to(torch.int32),
              "rope": rope, "q_out": torch.zeros((T + c["pad"], H, d), dtype=BF16, device="cuda")}
        s["cos"], s["sin"] = _tables(T + 64, rot)
        total = R * blocks + 3
        for n in "kv":
            if c["q4"]:
                s[n + "_cache"] = torch.zeros((total, Hkv, bs, d // 2), dtype=torch.uint8, device="cuda")
                s[n + "_scale"] = torch.zeros((total, Hkv, bs, d // 64, 2), dtype=BF16, device="cuda")
                s[n + "_values"] = torch.zeros((T + c["pad"], Hkv, d), dtype=BF16, device="cuda")
            else:
                s[n + "_cache"] = torch.zeros((total, Hkv, bs, d), dtype=BF16, device="cuda")
        return s
    B, N = c["B"], c["N"]
    qkv = randn(B, N, H + 2 * Hkv, d).to(BF16)
    s["q"], s["k"] = (x.transpose(1, 2) for x in (qkv[:, :, :H], qkv[:, :, H:H + Hkv]))
    s["rope"] = torch.stack([_grid_positions(N, g) for _ in range(B)], 1)  # [3, B, N]
    s["cos"], s["sin"] = _tables(N + 64, rot)
    if c["op"] == "norm_rope_bwd":
        s["dq_out"], s["dk_out"] = randn(B, H, N, d).to(BF16), randn(B, Hkv, N, d).to(BF16)
    return s


def _prepare_extend(c, g):
    B, H, Hkv, d, bs = c["B"], c["H"], c["Hkv"], c["d"], c["bs"]
    lens, new = _lengths(c)
    length = torch.tensor(lens, device="cuda")
    count = -(-length // bs)
    width = max(1, -(-c["longest"] // bs))
    total = sum(-(-n // bs) for n in lens) + 3
    order = torch.randperm(total, generator=g, device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    before = (count.cumsum(0) - count)[:, None]
    table = torch.where(slot < count[:, None], order[(before + slot).clamp(max=total - 1)], 0).to(torch.int32)
    used = torch.zeros((total, bs), dtype=torch.bool, device="cuda")
    token = torch.arange(width * bs, device="cuda")[None, :].expand(B, -1)
    live = token < length[:, None]
    used[table.long().gather(1, token // bs)[live], (token % bs)[live]] = True
    used = used[:, None, :, None]
    starts = torch.tensor([0] + new, device="cuda").cumsum(0)
    s = {"q": torch.randn((sum(new), H, d), generator=g, device="cuda").to(BF16), "table": table,
         "lens": length.to(torch.int32), "starts": starts.to(torch.int32)}
    for n in "kv":  # slots that hold no token hold whatever was there
        if c["q4"]:
            code = torch.randn((total, Hkv, bs, d), generator=g, device="cuda") * 3 + 8
            code = code.round().clamp(0, 15).to(torch.uint8)
            s[n + "_cache"] = code[..., 0::2] | (code[..., 1::2] << 4)
            pair = torch.stack([0.25 + 0.15 * torch.rand((total, Hkv, bs, d // 64), generator=g, device="cuda"),
                                0.15 * torch.randn((total, Hkv, bs, d // 64), generator=g, device="cuda")], -1)
            s[n + "_scale"] = torch.where(used[..., None], pair, float("nan")).to(BF16)
        else:
            x = torch.randn((total, Hkv, bs, d), generator=g, device="cuda")
            s[n + "_cache"] = torch.where(used, _keys(x, g) if n == "k" else x, float("nan")).to(BF16)
    return s


# --------------------------------------------------------------- plain forms

def _norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([both, x[..., rot:]], -1)


def _prepared(x, w, cos, sin, c):
    return _rotate(_norm(x, w), cos, sin, c["interleaved"])


def _angles(s, rope):
    """cos and sin [..., rot/2] of tokens with positions rope [3, ...]: each pair's of its own axis."""
    rows = rope.long()[s["axis_of_pair"]].movedim(0, -1)
    pair = torch.arange(rows.shape[-1], device="cuda")
    return s["cos"][rows, pair], s["sin"][rows, pair]


def _plain_norm_rope(s):
    c = s["case"]
    cos, sin = (t[:, None] for t in _angles(s, s["rope"]))
    return {"q": _prepared(s["q"].float(), s["q_weight"], cos, sin, c).to(BF16),
            "k": _prepared(s["k"].float(), s["k_weight"], cos, sin, c).to(BF16)}


def _back(dy, x, w, cos, sin, c):
    """Gradients of the norm and rotation of x: dx, dw."""
    g = _rotate(dy, cos, -sin, c["interleaved"])
    if w is None:
        return g, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    h = g * w.to(x.dtype)
    dw = (g * (x * r)).sum((0, 1, 2), dtype=torch.float64)
    return r * (h - x * (r * r * (h * x).mean(-1, keepdim=True))), dw


def _plain_norm_rope_bwd(s):
    c = s["case"]
    cos, sin = (t[:, None] for t in _angles(s, s["rope"]))
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
    cos, sin = (t[:, None] for t in _angles(s, s["rope"][:, :n]))
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


def _gathered(s, name, length):
    """[B, Hkv, length, d] values of the first `length` tokens of each request."""
    c = s["case"]
    token = torch.arange(length, device="cuda")
    block, slot = s["table"][:, token // c["bs"]].long(), token % c["bs"]
    rows = s[name + "_cache"][block, :, slot]
    if c["q4"]:
        code = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float()
        # read back as bf16, the values held
        return _held(code, s[name + "_scale"][block, :, slot].float()).to(BF16).float().transpose(1, 2)
    return rows.float().transpose(1, 2)


def _plain_extend(s):
    """The whole batch at once, requests padded to the longest."""
    c = s["case"]
    B, H, Hkv, d, longest, most = c["B"], c["H"], c["Hkv"], c["d"], c["longest"], c["new_most"]
    T = s["q"].shape[0]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    dead = (torch.arange(longest, device="cuda")[None, :] >= lens[:, None])[:, None, :, None]
    keys = _gathered(s, "k", longest).masked_fill(dead, 0.0)
    values = _gathered(s, "v", longest).masked_fill(dead, 0.0)
    i = torch.arange(most, device="cuda")
    row = (starts[:-1, None] + i).clamp(max=max(0, T - 1))  # [B, most]
    live = i < new[:, None]
    q = s["q"][row].float().view(B, most, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, most, d]
    scores = torch.matmul(q.reshape(B, Hkv, -1, d), keys.transpose(2, 3)).mul_(d ** -0.5)
    sight = (lens - new)[:, None] + i  # the last key each token sees
    hidden = torch.arange(longest, device="cuda") > sight[:, :, None]  # [B, most, longest]
    scores = scores.view(B, Hkv, H // Hkv, most, longest).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, longest), values).view(B, Hkv, -1, most, d)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    back = lambda x: x.permute(0, 3, 1, 2, *range(4, x.dim())).flatten(2, 3)[live]  # noqa: E731
    return {"o": back(o).to(BF16), "lse": back(lse)}


# ---------------------------------------------------------------------- runs

def _own_run(s):
    import exact_tiled_attention_24_gb300 as fa
    c = s["case"]
    if c["op"] == "extend":
        if c["q4"]:
            o, lse = fa.extend_paged_q4(s["q"], s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"], s["table"],
                                        s["lens"], s["starts"])
        else:
            o, lse = fa.extend_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["starts"])
        return {"o": o, "lse": lse}
    common = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"], axes=s["axes"])
    if c["op"] == "norm_rope":
        q, k = fa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["rope"], **common)
        return {"q": q, "k": k}
    if c["op"] == "norm_rope_bwd":
        dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["cos"], s["sin"],
                                               positions=s["rope"], **common)
        return {"dq": dq, "dk": dk} if dqw is None else {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    common |= dict(requests=s["requests"], rope_positions=s["rope"], cos=s["cos"], sin=s["sin"], q=s["q"],
                   q_out=s["q_out"])
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
    if op == "extend":
        return _plain_extend(state)
    if op == "norm_rope":
        return _plain_norm_rope(state)
    if op == "norm_rope_bwd":
        return _plain_norm_rope_bwd(state)
    return _plain_append(state)


# ------------------------------------------------------------- in 64 bits

def _exact_turn(s, rope):
    """e^(i angle) of each token's pairs, [..., pairs] complex: axis by axis."""
    out = None
    for axis in range(rope.shape[0]):
        rows = rope[axis].long()
        turn = torch.complex(s["cos"].double()[rows], s["sin"].double()[rows])
        mine = s["axis_of_pair"] == axis
        out = torch.where(mine, turn, torch.zeros_like(turn) if out is None else out)
    return out


def _exact_turned(x, w, turn, c):
    """Norm (w given), then each pair as a complex number times `turn`."""
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    rot = 2 * turn.shape[-1]
    order = torch.arange(rot, device="cuda")
    order = order.view(-1, 2) if c["interleaved"] else order.view(2, -1).t()
    y = x.clone()
    y[..., order] = torch.view_as_real(torch.view_as_complex(x[..., order].contiguous()) * turn)
    return y


def _exact_append(s):
    c, n, bs = s["case"], s["case"]["T"], s["case"]["bs"]
    position, request = s["positions"][:n].long(), s["requests"][:n].long()
    turn = _exact_turn(s, s["rope"][:, :n])[:, None]
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


def _exact_extend(s):
    c = s["case"]
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (length, new) in enumerate(zip(*_lengths(c))):
        rows = slice(at, at + new)
        at += new
        if length == 0 or new == 0:
            continue
        blocks = s["table"][b, :-(-length // c["bs"])].long()
        held = []
        for name in "kv":
            x = s[name + "_cache"][blocks].transpose(1, 2).flatten(0, 1)[:length]
            if c["q4"]:
                pair = s[name + "_scale"][blocks].transpose(1, 2).flatten(0, 1)[:length].double()[..., None]
                code = torch.empty((length, Hkv, d), dtype=torch.float64, device="cuda")
                code[..., 0::2], code[..., 1::2] = (x % 16).double(), torch.div(x, 16, rounding_mode="floor").double()
                x = (pair[..., 1, :] + pair[..., 0, :] * (code.view(length, Hkv, -1, 64) - 8)).reshape(length, Hkv, d)
                x = x.to(BF16)  # read back rounded: 64 bits hold the sum exactly, so this is its one rounding
            held.append(x.double())
        far = torch.arange(length, device="cuda")[None, :] > length - new + torch.arange(new, device="cuda")[:, None]
        for h in range(H):
            x = s["q"][rows, h].double() @ held[0][:, h // (H // Hkv)].t() / math.sqrt(d)
            x = x.masked_fill_(far, -math.inf)
            lse[rows, h] = torch.logsumexp(x, 1)
            o[rows, h] = torch.exp(x - lse[rows, h, None]) @ held[1][:, h // (H // Hkv)]
    return {"o": o, "lse": lse}


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "extend":
        return _exact_extend(s)
    turn = _exact_turn(s, s["rope"])[:, None]
    out = {}
    for name in "qk":
        x, w = s[name].double(), s[name + "_weight"]
        if c["op"] == "norm_rope":
            out[name] = _exact_turned(x, w, turn, c)
            continue
        g = _exact_turned(s["d" + name + "_out"].double(), None, turn.conj().resolve_conj(), c)
        if w is not None:  # y = u w with u = x / |x|rms: du = g w, less its part along u
            rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            u = x / rms
            out["d" + name + "_weight"] = (g * u).sum((0, 1, 2))
            g = g * w.double()
            g = (g - u * (g * u).mean(-1, keepdim=True)) / rms
        out["d" + name] = g
    return out
