"""Refusal of unknown bits beside FA_ZERO_SKIPPED in an append's weight_fp32,
and which calls of the binding set it (a fake library), on CPU."""
import pytest

import exact_tiled_attention_24_gb300 as fa
from exact_tiled_attention_24_gb300 import build as fabuild
from test_binding_checks import F32, I32, META, FakeLib, m  # noqa: F401

PTR = 0x10000


@pytest.mark.parametrize("entry", ["fa_append_paged", "fa_append_paged_q4"])
def test_unknown_bits_are_refused(entry):
    fabuild.build()
    row = (PTR, 1024, 128)

    def call(w32, k=row):
        args = fa._APPEND_ARGS.pack(*row, *k, *row, *row, *[PTR] * 13, 5, 3, 4, 2, 128, 10, 16, 8, 128, 64, w32, 0, 1e-6)
        return getattr(fa.lib(), entry)(args, None)

    for w32 in (4, 5, 6, -1, 1 << 30):
        assert call(w32) == 1, w32
    off = (PTR + 8, 1024, 128)
    for w32 in (0, 1, 2, 3):           # past that check: the next one refuses
        assert call(w32, k=off) == 3, w32


def test_the_binding_sets_it_for_outputs_it_makes(monkeypatch):
    packed = []

    class Lib(FakeLib):
        def __getattr__(self, name):
            entry = super().__getattr__(name)
            return lambda args, stream: packed.append(fa._APPEND_ARGS.unpack(args)[-3]) or entry(args, stream)

    monkeypatch.setattr(fa, "_DEVICE_TYPE", "meta")
    monkeypatch.setattr(fa, "lib", lambda L=Lib(): L)
    monkeypatch.setattr(fa, "_stream", lambda device: None)
    q, k, v = m(3, 4, 128), m(3, 2, 128), m(3, 2, 128)
    cache, table, pos = (m(7, 2, 16, 128), m(7, 2, 16, 128)), m(3, 4, dtype=I32), m(3, dtype=I32)
    w, w32 = m(128), m(128, dtype=F32)
    fa.append_paged(k, v, *cache, table, pos)
    fa.append_paged(k, v, *cache, table, pos, q=q)
    fa.append_paged(k, v, *cache, table, pos, q=q, q_out=q)
    fa.append_paged(k, v, *cache, table, pos, q=q, q_weight=w, k_weight=w)
    fa.append_paged(k, v, *cache, table, pos, q=q, q_weight=w32, k_weight=w32)
    fa.append_paged(k, v, *cache, table, pos, q=q, q_out=q, q_weight=w32, k_weight=w32)
    assert packed == [0, 2, 0, 2, 3, 1]
