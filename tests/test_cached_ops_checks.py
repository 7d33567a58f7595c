"""Argument checks, on CPU, of the norm and rotation calls, the paged appends
and the 4-bit decode: by the library (bad arguments are refused before any
CUDA call) and by the binding (a fake library, tensors without storage)."""
import struct

import pytest
import torch

import exact_tiled_attention_24_gb300 as fa
from exact_tiled_attention_24_gb300 import build as fabuild
from test_binding_checks import F32, I32, fake, m, rejects  # noqa: F401

FAKE, MIS, NUL = 0x10000, 0x10008, 0
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 6


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def heads(ptr=FAKE, sb=4096, sh=128, sn=1024):
    return ptr, sb, sh, sn


def tokens(ptr=FAKE, st=1024, sh=128):
    return ptr, st, sh


NO_HEADS, NO_TOKENS = (0, 0, 0, 0), (0, 0, 0)


def test_norm_rope_refusals(L):
    def call(q=heads(), k=heads(), qo=heads(), ko=heads(), cos=FAKE, sin=FAKE, pos=FAKE, per=0, qw=FAKE, kw=FAKE,
             w32=0, B=1, H=4, Hkv=2, N=16, d=128, rot=128, n_pos=64, eps=1e-6):
        return L.fa_qk_norm_rope(fa._NORM_ROPE_ARGS.pack(*q, *k, *qo, *ko, cos, sin, pos, qw, kw, B, H, Hkv, N, d, rot,
                                                         n_pos, per, w32, 0, eps), None)

    assert L.fa_qk_norm_rope(None, None) == INVALID
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: heads(ptr=0)}) == INVALID
    assert call(q=heads(sn=-128)) == INVALID
    assert call(cos=NUL) == INVALID and call(sin=NUL) == INVALID and call(n_pos=0) == INVALID
    assert call(qw=NUL) == INVALID and call(kw=NUL) == INVALID       # one weight without the other
    assert call(qw=NUL, kw=NUL, rot=0) == INVALID                    # nothing to do
    assert call(w32=2) == INVALID and call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(pos=NUL, N=65) == INVALID                            # fewer angles than tokens
    assert call(rot=-16) == INVALID
    for size in ("B", "H", "Hkv", "N"):
        assert call(**{size: 0}) == INVALID
    assert call(d=96) == UNSUPPORTED and call(rot=24) == UNSUPPORTED and call(rot=144) == UNSUPPORTED
    assert call(d=64, rot=128) == UNSUPPORTED and call(H=70000) == UNSUPPORTED
    assert call(B=1 << 16, H=1 << 10, N=1 << 10) == UNSUPPORTED
    for bad in (dict(q=heads(ptr=MIS)), dict(k=heads(sh=132)), dict(qo=heads(sb=4)), dict(ko=heads(sn=1)),
                dict(cos=MIS), dict(sin=MIS), dict(qw=MIS), dict(kw=MIS), dict(pos=0x10002)):
        assert call(**bad) == MISALIGNED, bad


def test_norm_rope_bwd_refusals(L):
    ws = L.fa_qk_norm_rope_bwd_workspace_bytes(1, 16, 128)
    assert ws > 0 and ws % (2 * 128 * 4) == 0
    assert L.fa_qk_norm_rope_bwd_workspace_bytes(0, 16, 128) == 0
    assert L.fa_qk_norm_rope_bwd_workspace_bytes(1, 16, 96) == 0
    assert L.fa_qk_norm_rope_bwd_workspace_bytes(1 << 16, 1 << 16, 64) == 0

    def call(dqo=heads(), dko=heads(), q=heads(), k=heads(), dq=heads(), dk=heads(), dqw=FAKE, dkw=FAKE, qw=FAKE,
             kw=FAKE, work=FAKE, ws_bytes=ws, d=128, rot=128):
        a = fa._NORM_ROPE_ARGS.pack(*q, *k, *dqo, *dko, FAKE, FAKE, NUL, qw, kw, 1, 4, 2, 16, d, rot, 16, 0, 0, 0, 1e-6)
        return L.fa_qk_norm_rope_bwd(a, fa._NORM_ROPE_GRADS.pack(*dq, *dk, dqw, dkw, work, ws_bytes), None)

    assert L.fa_qk_norm_rope_bwd(None, None, None) == INVALID
    assert call(dqo=NO_HEADS) == INVALID and call(q=NO_HEADS) == INVALID and call(dk=NO_HEADS) == INVALID
    assert call(dq=heads(ptr=0)) == INVALID and call(dq=heads(sb=-8)) == INVALID
    assert call(dqw=NUL) == INVALID and call(dkw=NUL) == INVALID and call(kw=NUL) == INVALID
    assert call(work=NUL) == WORKSPACE and call(ws_bytes=ws - 1) == WORKSPACE
    assert call(d=80) == UNSUPPORTED and call(rot=8) == UNSUPPORTED
    assert call(work=MIS) == MISALIGNED and call(dqw=MIS) == MISALIGNED and call(dk=heads(sh=4)) == MISALIGNED
    # without weights neither q, k, the weight gradients nor a workspace are asked for
    assert call(q=NO_HEADS, k=NO_HEADS, qw=NUL, kw=NUL, dqw=NUL, dkw=NUL, work=NUL, dq=heads(ptr=MIS)) == MISALIGNED
    assert call(q=NO_HEADS, k=NO_HEADS, qw=NUL, kw=NUL, rot=0) == INVALID


@pytest.mark.parametrize("q4", [False, True])
def test_append_refusals(L, q4):
    def call(q=tokens(), k=tokens(), v=tokens(), qo=tokens(), kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, kv=FAKE, vv=FAKE,
             table=FAKE, pos=FAKE, req=FAKE, cos=FAKE, sin=FAKE, qw=FAKE, kw=FAKE, w32=0, T=5, B=3, H=4, Hkv=2, d=128,
             num_blocks=10, bs=16, max_blocks=8, rot=128, n_pos=64, eps=1e-6):
        args = fa._APPEND_ARGS.pack(*q, *k, *v, *qo, kc, vc, ks, vs, kv, vv, table, pos, req, cos, sin, qw, kw, T, B,
                                    H, Hkv, d, num_blocks, bs, max_blocks, rot, n_pos, w32, 0, eps)
        return (L.fa_append_paged_q4 if q4 else L.fa_append_paged)(args, None)

    assert L.fa_append_paged(None, None) == INVALID and L.fa_append_paged_q4(None, None) == INVALID
    for bad in (dict(k=NO_TOKENS), dict(v=NO_TOKENS), dict(k=tokens(ptr=0)), dict(kc=NUL), dict(vc=NUL), dict(table=NUL),
                dict(pos=NUL), dict(q=NO_TOKENS), dict(qo=NO_TOKENS), dict(v=tokens(st=-8)),
                dict(q=NO_TOKENS, qo=NO_TOKENS), dict(qw=NUL), dict(kw=NUL), dict(T=0), dict(B=0), dict(H=0), dict(Hkv=0),
                dict(num_blocks=0), dict(bs=0), dict(max_blocks=0), dict(req=NUL), dict(cos=NUL), dict(rot=-16),
                dict(n_pos=0), dict(eps=float("inf"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(rot=8), dict(rot=144), dict(H=20000), dict(max_blocks=1 << 27),
                dict(num_blocks=1 << 28, bs=8), dict(num_blocks=1 << 30, Hkv=64)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(k=tokens(ptr=MIS)), dict(v=tokens(sh=4)), dict(q=tokens(st=12)), dict(qo=tokens(ptr=MIS)),
                dict(kc=MIS), dict(vc=MIS), dict(cos=MIS), dict(kw=MIS), dict(pos=0x10001), dict(req=0x10002),
                dict(table=0x10003)):
        assert call(**bad) == MISALIGNED, bad
    if q4:
        for bad in (dict(ks=NUL), dict(vs=NUL), dict(kv=NUL), dict(vv=NUL)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(ks=MIS), dict(vs=MIS), dict(kv=MIS), dict(vv=MIS)):
            assert call(**bad) == MISALIGNED, bad


def test_decode_q4_refusals(L):
    ws = L.fa_decode_workspace_bytes(2, 8, 128, 4)

    def call(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=FAKE, work=FAKE,
             ws_bytes=ws, B=2, H=8, Hkv=2, d=128, num_blocks=10, bs=16, max_blocks=8, scale=0.1, S=4):
        args = fa._DECODE_Q4_ARGS.pack(q, kc, ks, vc, vs, table, lens, o, lse, work, ws_bytes, B, H, Hkv, d, num_blocks,
                                       bs, max_blocks, S, scale)
        return L.fa_decode_paged_q4(args, None)

    assert L.fa_decode_paged_q4(None, None) == INVALID
    for name in ("q", "kc", "ks", "vc", "vs", "table", "lens", "o", "lse"):
        assert call(**{name: NUL}) == INVALID, name
    for bad in (dict(B=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(S=0), dict(bs=0), dict(num_blocks=0),
                dict(max_blocks=0), dict(scale=0.0), dict(scale=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(B=70000), dict(S=5000), dict(max_blocks=1 << 27), dict(num_blocks=1 << 28, bs=8)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(work=NUL) == WORKSPACE and call(ws_bytes=ws - 1) == WORKSPACE
    assert call(work=NUL, ws_bytes=0, S=1, q=MIS) == MISALIGNED   # one split asks for no workspace
    for name in ("q", "kc", "ks", "vc", "vs", "o", "work"):
        assert call(**{name: MIS}) == MISALIGNED, name
    for name in ("table", "lens", "lse"):
        assert call(**{name: 0x10002}) == MISALIGNED, name


def test_split_choice(L):
    f = L.fa_decode_q4_splits
    assert f(1, 8, 3, 16, 8) == 0 and f(0, 8, 2, 16, 8) == 0 and f(1, 8, 2, 0, 8) == 0
    assert f(1, 8, 2, 16, 1) == 1                 # one block: nothing to split
    assert f(4096, 32, 8, 16, 512) == 1           # enough requests to fill the GPU
    assert 1 < f(1, 32, 8, 16, 8192) <= 4096      # one long context
    assert f(1, 1, 1, 128, 1 << 22) <= 4096


def test_binding_norm_rope(fake):  # noqa: F811
    B, H, Hkv, N, d = 2, 4, 2, 8, 64
    qkv = m(B, N, H + 2 * Hkv, d)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
    cos, sin = m(20, 32, dtype=F32), m(20, 32, dtype=F32)
    w = m(d)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, q_weight=w, k_weight=w)
    assert qo.shape == (B, H, N, d) and qo.is_contiguous() and ko.shape == (B, Hkv, N, d)
    fa.qk_norm_rope(q, k, cos, sin, positions=m(B, N, dtype=I32), q_out=q, k_out=k)      # in place
    fa.qk_norm_rope(q, k, q_weight=m(d, dtype=F32), k_weight=m(d, dtype=F32))
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(qo, ko, q, k, cos, sin, positions=m(N, dtype=I32), q_weight=w, k_weight=w,
                                           workspace=m(1 << 16, dtype=torch.uint8))
    assert dq.shape == qo.shape and dqw.shape == (d,) and dqw.dtype == F32
    assert fa.qk_norm_rope_bwd(qo, ko, None, None, cos, sin)[2:] == (None, None)
    assert fake.calls.count("fa_qk_norm_rope") == 3 and fake.calls.count("fa_qk_norm_rope_bwd") == 2
    for bad in (dict(q_weight=w), dict(cos=cos, q_weight=w, k_weight=w), dict(q_weight=w, k_weight=m(d, dtype=F32)),
                dict(q_weight=m(d + 1), k_weight=w), {}, dict(cos=m(4, 32, dtype=F32), sin=m(4, 32, dtype=F32)),
                dict(cos=cos, sin=m(19, 32, dtype=F32)), dict(cos=cos, sin=sin, positions=m(N + 1, dtype=I32)),
                dict(cos=cos, sin=sin, positions=m(B, N, dtype=torch.int64)),
                dict(cos=cos, sin=sin, q_out=m(B, H, N, d + 8)), dict(cos=cos, sin=sin, k_out=m(B, Hkv, N, d, dtype=F32)),
                dict(cos=cos, sin=sin, q_out=m(B, 1, N, d).expand(B, H, N, d)),                 # overlapping rows
                dict(cos=cos, sin=sin, q_out=torch.empty(B, H, N, d, dtype=torch.bfloat16))):  # another device
        rejects(fake, fa.qk_norm_rope, q, k, **bad)
    rejects(fake, fa.qk_norm_rope, m(B, H, d, N).transpose(2, 3), k, cos, sin)     # d not contiguous
    rejects(fake, fa.qk_norm_rope, m(B, H, N, d + 4)[..., :d], k, cos, sin)        # rows off 16-byte boundaries
    rejects(fake, fa.qk_norm_rope, q, m(B, Hkv, N + 1, d), cos, sin)
    rejects(fake, fa.qk_norm_rope_bwd, qo, ko, q, k, cos, sin, q_weight=w, k_weight=w, dq=m(B, H, N, 2 * d))
    rejects(fake, fa.qk_norm_rope_bwd, qo, m(B, H, N, d), q, k, cos, sin, q_weight=w, k_weight=w)
    rejects(fake, fa.qk_norm_rope_bwd, qo, ko, q, k, cos, sin, q_weight=w, k_weight=w,
            workspace=torch.empty(1 << 16, dtype=torch.uint8))


def test_binding_appends(fake):  # noqa: F811
    T, H, Hkv, d, nb, bs, B, mb = 5, 4, 2, 128, 7, 16, 3, 4
    qkv = m(T, H + 2 * Hkv, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    kc, vc = m(nb, Hkv, bs, d), m(nb, Hkv, bs, d)
    codes, pairs = m(nb, Hkv, bs, d // 2, dtype=torch.uint8), m(nb, Hkv, bs, d // 64, 2)
    table, pos, req = m(B, mb, dtype=I32), m(T, dtype=I32), m(T, dtype=I32)
    cos, sin = m(64, 64, dtype=F32), m(64, 64, dtype=F32)
    assert fa.append_paged(k, v, kc, vc, table, pos, req) is None
    out = fa.append_paged(k, v, kc, vc, table, pos, req, cos, sin, q=q)
    assert out.shape == (T, H, d)
    fa.append_paged(k[:3], v[:3], kc, vc, table, pos[:3], None, cos, sin, k_weight=m(d))   # a step; keys' norm alone
    fa.append_paged_q4(k, v, codes, pairs, codes, pairs, table, pos, req, cos, sin, q=q, q_out=q,
                       k_values=m(T, Hkv, d), v_values=m(T, Hkv, d))
    assert [c for c in fake.calls] == ["fa_append_paged"] * 3 + ["fa_append_paged_q4"]
    both = ((fa.append_paged, (kc, vc)), (fa.append_paged_q4, (codes, pairs, codes, pairs)))
    for fn, cache in both:
        rejects(fake, fn, k, v, *cache, table, pos)                       # 5 tokens, 3 requests
        rejects(fake, fn, k, v[:4], *cache, table, pos, req)
        rejects(fake, fn, k, v, *cache, table, pos[:4], req)
        rejects(fake, fn, k, v, *cache, table, pos, m(T, dtype=torch.int64))
        rejects(fake, fn, k, v, *cache, table[:, ::2], pos, req)
        rejects(fake, fn, k, v, *cache, torch.zeros(B, mb, dtype=I32), pos, req)
        rejects(fake, fn, k, v, *cache, table, pos, req, cos=cos)
        rejects(fake, fn, k, v, *cache, table, pos, req, q_weight=m(d))
        rejects(fake, fn, k, v, *cache, table, pos, req, q=q, q_weight=m(d))
        rejects(fake, fn, k, v, *cache, table, pos, req, q_out=m(T, H, d))
        rejects(fake, fn, k, v, *cache, table, pos, req, q=m(T, H, d // 2))
        rejects(fake, fn, k, v, *cache, table, pos, req, q=q, q_out=m(T, 1, d).expand(T, H, d))
        rejects(fake, fn, k, m(T, Hkv, d + 4)[..., :d], *cache, table, pos, req)
    rejects(fake, fa.append_paged, k, v, kc, m(nb, Hkv, bs + 1, d), table, pos, req)
    rejects(fake, fa.append_paged, k, v, kc[:, :1], vc[:, :1], table, pos, req)
    rejects(fake, fa.append_paged, k, v, kc.transpose(1, 2), vc.transpose(1, 2), table, pos, req)
    rejects(fake, fa.append_paged_q4, k, v, codes, m(nb, Hkv, bs, d // 64), codes, pairs, table, pos, req)
    rejects(fake, fa.append_paged_q4, k, v, kc, pairs, vc, pairs, table, pos, req)
    rejects(fake, fa.append_paged_q4, k, v, codes, pairs, codes, pairs, table, pos, req, k_values=m(T, Hkv, d))


def test_binding_decode_q4(fake):  # noqa: F811
    B, H, Hkv, d, nb, bs, mb = 3, 8, 2, 128, 12, 16, 5
    q = m(B, H, d)
    codes, pairs = m(nb, Hkv, bs, d // 2, dtype=torch.uint8), m(nb, Hkv, bs, d // 64, 2)
    table, lens = m(B, mb, dtype=I32), m(B, dtype=I32)
    good = (q, codes, pairs, codes, pairs, table, lens)
    o, lse = fa.decode_paged_q4(*good, n_splits=2)
    assert o.shape == q.shape and lse.shape == (B, H)
    for i, bad in ((0, m(B, H, d, dtype=F32)), (0, q.transpose(0, 1)), (1, m(nb, Hkv, bs, d, dtype=torch.uint8)),
                   (2, m(nb, Hkv, bs, d // 64, 2, dtype=F32)), (3, m(nb, Hkv, bs + 1, d // 2, dtype=torch.uint8)),
                   (4, m(nb, Hkv, bs, 1, 2)), (5, m(B + 1, mb, dtype=I32)), (5, m(B, mb, dtype=torch.int64)),
                   (6, m(B, 2, dtype=I32)[:, 0]), (6, torch.zeros(B, dtype=I32))):
        args = list(good)
        args[i] = bad
        rejects(fake, fa.decode_paged_q4, *args, n_splits=2)
    rejects(fake, fa.decode_paged_q4, *good, n_splits=2, out=m(B, H, d - 8))
    rejects(fake, fa.decode_paged_q4, *good, n_splits=2, lse=m(B, H))
    rejects(fake, fa.decode_paged_q4, *good, n_splits=2, workspace=torch.empty(1 << 16, dtype=torch.uint8))


def test_host_tensors_refused(monkeypatch):
    def no_lib():
        raise AssertionError("library called")
    monkeypatch.setattr(fa, "lib", no_lib)
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    cos, sin = fa.rope_tables(4, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x, cos, sin)
    with pytest.raises(ValueError):
        fa.append_paged(x[0], x[0], x, x, torch.zeros(4, 4, dtype=I32), torch.zeros(2, dtype=I32))
    with pytest.raises(ValueError):
        fa.decode_paged_q4(x[0], x, x, x, x, torch.zeros(4, 4, dtype=I32), torch.zeros(2, dtype=I32))


def test_rope_tables_far_positions():
    import math
    cos, sin = fa.rope_tables(200_001, 64, base=1e4, device="cpu")
    for i in (0, 1, 31):
        a = 200_000 * 1e4 ** (-2 * i / 64)
        assert abs(float(cos[200_000, i]) - math.cos(a)) < 1e-7 and abs(float(sin[200_000, i]) - math.sin(a)) < 1e-7
    for bad in ((0, 64), (4, 0), (4, 7)):
        with pytest.raises(ValueError):
            fa.rope_tables(*bad, device="cpu")


def test_structs_match_the_header(tmp_path):
    """The packed argument structs have the C structs' layout."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text('''
#include <stdio.h>
#include "fa.h"
#define AT(s, f) printf("%zu ", offsetof(s, f));
int main(void) {
  AT(fa_norm_rope_args, q_out) AT(fa_norm_rope_args, cos) AT(fa_norm_rope_args, k_weight)
  AT(fa_norm_rope_args, B) AT(fa_norm_rope_args, interleaved) AT(fa_norm_rope_args, eps)
  AT(fa_norm_rope_grads, dq_weight) AT(fa_norm_rope_grads, ws_bytes)
  AT(fa_append_args, q_out) AT(fa_append_args, k_cache) AT(fa_append_args, block_table) AT(fa_append_args, k_weight)
  AT(fa_append_args, T) AT(fa_append_args, n_pos) AT(fa_append_args, eps)
  AT(fa_decode_q4_args, ws_bytes) AT(fa_decode_q4_args, B) AT(fa_decode_q4_args, n_splits) AT(fa_decode_q4_args, scale)
  return 0;
}
''')
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    at = lambda fmt: struct.calcsize("@" + fmt)  # noqa: E731
    h, t = "Pqqq", "Pqq"
    a, b = 4 * h, 4 * t
    assert got == [at(2 * h), at(a), at(a + "4P"), at(a + "5P"), at(a + "5P9i"), at(a + "5P10i"), at(2 * h), at(2 * h + "3P"),
                   at(3 * t), at(b), at(b + "6P"), at(b + "12P"), at(b + "13P"), at(b + "13P9i"), at(b + "13P12i"),
                   at("10P"), at("10PN"), at("10PN7i"), at("10PN8i")]
