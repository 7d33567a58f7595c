"""What the `axes` of rotations and appends may be, on CPU (a fake library,
tensors without storage): numbers of axes, one a pair, in any sequence. A single
number is none, though bytes(n) makes n zeros of it."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_24_gb300 as fa
from test_binding_checks import F32, I32, fake, m, rejects  # noqa: F401


def calls():
    B, H, Hkv, N, d, T, nb, bs, mb = 2, 4, 2, 8, 64, 5, 7, 16, 4
    cos, sin = m(20, 32, dtype=F32), m(20, 32, dtype=F32)
    pos = m(3, N, dtype=I32)
    yield lambda axes: fa.qk_norm_rope(m(B, H, N, d), m(B, Hkv, N, d), cos, sin, positions=pos, axes=axes)
    yield lambda axes: fa.qk_norm_rope_bwd(m(B, H, N, d), m(B, Hkv, N, d), None, None, cos, sin, positions=pos, axes=axes)
    table, slot, req = m(B, mb, dtype=I32), m(T, dtype=I32), m(T, dtype=I32)
    codes, pairs = m(nb, Hkv, bs, d // 2, dtype=torch.uint8), m(nb, Hkv, bs, d // 64, 2)
    for fn, cache in ((fa.append_paged, (m(nb, Hkv, bs, d),) * 2), (fa.append_paged_q4, (codes, pairs, codes, pairs))):
        yield lambda axes, fn=fn, cache=cache: fn(m(T, Hkv, d), m(T, Hkv, d), *cache, table, slot, req, cos, sin,
                                                  rope_positions=m(3, T, dtype=I32), axes=axes)


def test_a_number_is_no_assignment(fake):  # noqa: F811
    for call in calls():
        for bad in (32, np.int64(32), True, 0, 1.5, "0" * 32, [0.0] * 32, [None] * 32, torch.tensor(32)):
            rejects(fake, call, bad)


def test_sequences_of_axis_numbers(fake):  # noqa: F811
    want = fa.rope_axes((8, 12, 12), in_turn=True)
    for form in (want, bytearray(want), list(want), tuple(want), np.frombuffer(want, np.uint8),
                 np.array(list(want), np.int32), torch.tensor(list(want))):
        assert fa._pack_axes(form, torch.zeros((3, 1), dtype=I32), 3, 64)[-64:-32] == want
    for call in calls():
        call(list(want))
    assert len(fake.calls) == 4


@pytest.mark.parametrize("bad", [b"\0" * 31, b"\0" * 33, [0, 300] * 16, [-1] * 32, []])
def test_wrong_numbers(fake, bad):  # noqa: F811
    for call in calls():
        rejects(fake, call, bad)
