"""Argument checks, on CPU, of the chunk attention and of rotations with
several position axes: by the library (bad arguments are refused before any
CUDA call) and by the binding (a fake library, tensors without storage)."""
import os
import shutil
import struct
import subprocess

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


@pytest.mark.parametrize("q4", [False, True])
def test_extend_refusals(L, q4):
    ws = L.fa_extend_workspace_bytes(40, 3, 8, 2, 128, 16, 8)
    assert ws > 0

    def call(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, lens=FAKE, starts=FAKE, o=FAKE, lse=FAKE, work=FAKE,
             ws_bytes=ws, T=40, B=3, H=8, Hkv=2, d=128, num_blocks=20, bs=16, max_blocks=8, scale=0.1):
        args = fa._EXTEND_ARGS.pack(q, kc, ks, vc, vs, table, lens, starts, o, lse, work, ws_bytes, T, B, H, Hkv, d,
                                    num_blocks, bs, max_blocks, 1, 0, scale)
        return (L.fa_extend_paged_q4 if q4 else L.fa_extend_paged)(args, None)

    assert L.fa_extend_paged(None, None) == INVALID and L.fa_extend_paged_q4(None, None) == INVALID
    for name in ("q", "kc", "vc", "table", "lens", "starts", "o", "lse") + (("ks", "vs") if q4 else ()):
        assert call(**{name: NUL}) == INVALID, name
    for bad in (dict(T=0), dict(B=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(num_blocks=0), dict(bs=0),
                dict(max_blocks=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(T=1 << 28, H=16), dict(T=(1 << 30) + 1, H=1, Hkv=1), dict(B=(1 << 24) + 1),
                dict(H=16385, Hkv=1), dict(max_blocks=1 << 27), dict(num_blocks=1 << 28, bs=8),
                dict(num_blocks=1 << 30, bs=1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(work=NUL) == WORKSPACE and call(ws_bytes=15) == WORKSPACE
    for name in ("q", "kc", "vc", "o", "work") + (("ks", "vs") if q4 else ()):
        assert call(**{name: MIS}) == MISALIGNED, name
    for name in ("table", "lens", "starts", "lse"):
        assert call(**{name: 0x10002}) == MISALIGNED, name


def test_extend_workspace(L):
    f = L.fa_extend_workspace_bytes
    for bad in ((0, 1, 8, 2, 128, 16, 8), (4, 0, 8, 2, 128, 16, 8), (4, 1, 8, 3, 128, 16, 8), (4, 1, 8, 2, 96, 16, 8),
                (4, 1, 8, 2, 128, 0, 8), (4, 1, 8, 2, 128, 16, 0)):
        assert f(*bad) == 0, bad
    part = 256 * 129 * 4
    assert f(1, 1, 8, 2, 128, 16, 1) < 3 * part                              # one tile: one CTA, two parts at most
    assert f(32, 32, 32, 8, 128, 16, 512) <= 2 * 152 * (part + 64)           # one item a head: two parts a CTA
    assert f(1 << 17, 1, 32, 8, 128, 16, 1 << 13) <= 20 * 152 * (part + 64)  # however long the prompt and its prefix


def axes(pairs=(0,) * 64, n=3, positions=FAKE):
    return fa._ROPE_AXES.pack(positions, n, bytes(pairs))


def test_axes_refusals(L):
    h = lambda ptr=FAKE: (ptr, 4096, 128, 1024)  # noqa: E731
    t = (FAKE, 1024, 128)

    def norm(x, pos=NUL, rot=128, n_pos=8, q=FAKE):
        a = fa._NORM_ROPE_ARGS.pack(*h(q), *h(), *h(), *h(), FAKE, FAKE, pos, FAKE, FAKE, 1, 4, 2, 16, 128, rot, n_pos,
                                    0, 0, 0, 1e-6)
        g = fa._NORM_ROPE_GRADS.pack(*h(), *h(), FAKE, FAKE, FAKE, 1 << 30)
        got = {L.fa_qk_norm_rope_axes(a, x, None), L.fa_qk_norm_rope_axes_bwd(a, x, g, None)}
        assert len(got) == 1
        return got.pop()

    def append(x, rot=128, k=t):
        a = fa._APPEND_ARGS.pack(*t, *k, *t, *t, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                 5, 3, 4, 2, 128, 10, 16, 8, rot, 64, 0, 0, 1e-6)
        got = {L.fa_append_paged_axes(a, x, None), L.fa_append_paged_q4_axes(a, x, None)}
        assert len(got) == 1
        return got.pop()

    assert L.fa_qk_norm_rope_axes(None, axes(), None) == INVALID and L.fa_append_paged_axes(None, axes(), None) == INVALID
    third = [0, 1, 2] * 21 + [0]
    for call in (norm, append):
        assert call(None) == INVALID and call(axes(positions=NUL)) == INVALID
        assert call(axes(n=0)) == INVALID and call(axes(n=5)) == INVALID and call(axes(n=-1)) == INVALID
        assert call(axes(third, n=2)) == INVALID                 # a pair on an axis that is not there
        assert call(axes([0] * 63 + [3], n=3)) == INVALID
        assert call(axes(), rot=0) == INVALID
        assert call(axes(), rot=24) == UNSUPPORTED
        assert call(axes(third, positions=0x10002)) == MISALIGNED
    assert norm(axes(third), pos=FAKE) == INVALID                # positions given twice
    assert norm(axes(third), q=MIS) == MISALIGNED                # n_pos < N is no error here
    assert append(axes(third), k=(MIS, 1024, 128)) == MISALIGNED
    # pairs past rot/2 are not looked at
    assert append(axes([0] * 16 + [9] * 48), rot=32, k=(MIS, 1024, 128)) == MISALIGNED


def test_binding_extend(fake):  # noqa: F811
    T, B, H, Hkv, d, nb, bs, mb = 9, 3, 8, 2, 128, 12, 16, 5
    q, kc, vc = m(T, H, d), m(nb, Hkv, bs, d), m(nb, Hkv, bs, d)
    codes, pairs = m(nb, Hkv, bs, d // 2, dtype=torch.uint8), m(nb, Hkv, bs, d // 64, 2)
    rest = (m(B, mb, dtype=I32), m(B, dtype=I32), m(B + 1, dtype=I32))
    for fn, cache in ((fa.extend_paged, (kc, vc)), (fa.extend_paged_q4, (codes, pairs, codes, pairs))):
        o, lse = fn(q, *cache, *rest)
        assert o.shape == q.shape and lse.shape == (T, H) and lse.dtype == F32
        fn(q, *cache, *rest, causal=False, out=q, lse=lse, workspace=m(1 << 16, dtype=torch.uint8), scale=0.1)
        n = len(cache)
        good = (q, *cache, *rest)
        wrong = [(0, m(T, H, d, dtype=F32)), (0, m(H, T, d).transpose(0, 1)), (0, m(T, H, d, 1)), (0, m(T, H, 64)),
                 (1, m(nb, Hkv, bs, d, dtype=F32)), (1, cache[0].transpose(1, 2)), (n - 1, m(nb, Hkv, bs + 1, d // 2)),
                 (n + 1, m(B, mb, dtype=torch.int64)), (n + 1, m(B + 1, mb, dtype=I32)), (n + 1, m(mb, dtype=I32)),
                 (n + 2, m(B + 1, dtype=I32)), (n + 2, torch.zeros(B, dtype=I32)), (n + 3, m(B, dtype=I32)),
                 (n + 3, m(B + 1, 2, dtype=I32)[:, 0]), (n + 3, None), (1, None)]
        for i, bad in wrong:
            args = list(good)
            args[i] = bad
            rejects(fake, fn, *args)
        rejects(fake, fn, *good, out=m(T, H, d + 8))
        rejects(fake, fn, *good, lse=m(T, H))
        rejects(fake, fn, *good, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    assert [c for c in fake.calls if "workspace" not in c] == ["fa_extend_paged"] * 2 + ["fa_extend_paged_q4"] * 2


def test_binding_axes(fake):  # noqa: F811
    B, H, Hkv, N, d = 2, 4, 2, 8, 64
    q, k = m(B, H, N, d), m(B, Hkv, N, d)
    cos, sin = m(20, 32, dtype=F32), m(20, 32, dtype=F32)
    sec = fa.rope_axes((8, 12, 12))
    for pos in (m(3, N, dtype=I32), m(3, B, N, dtype=I32)):
        fa.qk_norm_rope(q, k, cos, sin, positions=pos, axes=sec)
        fa.qk_norm_rope_bwd(q, k, None, None, cos, sin, positions=pos, axes=sec)
    fa.qk_norm_rope(q, k, cos, sin, positions=m(1, N, dtype=I32), axes=[0] * 32)
    assert fake.calls == ["fa_qk_norm_rope_axes", "fa_qk_norm_rope_axes_bwd"] * 2 + ["fa_qk_norm_rope_axes"]
    for bad in (dict(axes=sec), dict(axes=sec, positions=m(N, dtype=I32)), dict(axes=sec[:-1], positions=m(3, N, dtype=I32)),
                dict(axes=sec, positions=m(3, N + 1, dtype=I32)), dict(axes=sec, positions=m(3, N, B, dtype=I32)),
                dict(axes=sec, positions=m(3, N)), dict(axes=[0, 300] * 16, positions=m(3, N, dtype=I32)),
                dict(axes=sec, positions=m(N, 3, dtype=I32).t())):
        rejects(fake, fa.qk_norm_rope, q, k, cos, sin, **bad)
    rejects(fake, fa.qk_norm_rope, q, k, q_weight=m(d), k_weight=m(d), positions=m(3, N, dtype=I32), axes=sec)
    del fake.calls[:]
    T, nb, bs, mb = 5, 7, 16, 4
    k, v, qt = m(T, Hkv, d), m(T, Hkv, d), m(T, H, d)
    table, pos, req = m(B, mb, dtype=I32), m(T, dtype=I32), m(T, dtype=I32)
    codes, pairs = m(nb, Hkv, bs, d // 2, dtype=torch.uint8), m(nb, Hkv, bs, d // 64, 2)
    for fn, cache in ((fa.append_paged, (m(nb, Hkv, bs, d), m(nb, Hkv, bs, d))),
                      (fa.append_paged_q4, (codes, pairs, codes, pairs))):
        args = (k, v, *cache, table, pos, req, cos, sin)
        fn(*args, q=qt, rope_positions=m(3, T, dtype=I32), axes=sec)
        fn(*args, rope_positions=pos)
        for bad in (dict(axes=sec), dict(axes=sec, rope_positions=pos), dict(rope_positions=m(3, T, dtype=I32)),
                    dict(axes=sec, rope_positions=m(3, T + 1, dtype=I32)), dict(axes=sec[1:], rope_positions=m(3, T, dtype=I32)),
                    dict(rope_positions=m(T, dtype=torch.int64)), dict(rope_positions=[0] * T)):
            rejects(fake, fn, *args, **bad)
        rejects(fake, fn, k, v, *cache, table, pos, req, rope_positions=pos)   # nothing to turn by
    assert fake.calls == ["fa_append_paged_axes"] * 2 + ["fa_append_paged_q4_axes"] * 2


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text('''
#include <stdio.h>
#include "fa.h"
#define AT(s, f) printf("%zu ", offsetof(s, f));
int main(void) {
  AT(fa_rope_axes, n_axes) AT(fa_rope_axes, pair_axis) printf("%zu ", sizeof(fa_rope_axes));
  AT(fa_extend_args, workspace) AT(fa_extend_args, ws_bytes) AT(fa_extend_args, T) AT(fa_extend_args, num_blocks)
  AT(fa_extend_args, causal) AT(fa_extend_args, scale) printf("%zu ", sizeof(fa_extend_args));
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
    assert got == [at("P"), at("Pi"), at("Pi64s0P"), at("10P"), at("11P"), at("11PN"), at("11PN5i"), at("11PN8i"),
                   at("11PN10i"), at("11PN10if0P")]
