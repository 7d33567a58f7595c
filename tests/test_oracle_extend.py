"""The fp64 definition of chunk attention, against what it has to satisfy; and
the axes that rope_axes deals out."""
import numpy as np
import pytest

import exact_tiled_attention_24_gb300 as fa
from oracle import attention_fwd_head, decode_paged, extend_paged


def cache(B, mb, Hkv, bs, d, seed):
    rng = np.random.default_rng(seed)
    table = rng.permutation(B * mb + 2)[:B * mb].reshape(B, mb)
    return (*rng.standard_normal((2, B * mb + 2, Hkv, bs, d)), table, rng)


def test_one_token_is_a_decode_step():
    K, V, table, rng = cache(3, 4, 2, 5, 16, 1)
    q, lens = rng.standard_normal((3, 4, 16)), np.array([1, 20, 13])
    o, lse, _ = extend_paged(q, K, V, table, lens, np.arange(4), 0.3)
    ro, rl = decode_paged(q, K, V, table, lens, 0.3)
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(lse, rl, atol=1e-13)


def test_chunks_are_the_causal_prompt():
    K, V, table, rng = cache(1, 5, 1, 7, 16, 2)
    q = rng.standard_normal((33, 2, 16))
    parts = [extend_paged(q[a:b], K, V, table, [b], [0, b - a], 0.25)[:2] for a, b in ((0, 1), (1, 20), (20, 33))]
    t = np.arange(33)
    k, v = (c[table[0][t // 7], 0, t % 7] for c in (K, V))
    for h in range(2):
        ro, rl = attention_fwd_head(q[:, h], k, v, 0.25, True)
        np.testing.assert_allclose(np.concatenate([p[0] for p in parts])[:, h], ro, atol=1e-13)
        np.testing.assert_allclose(np.concatenate([p[1] for p in parts])[:, h], rl, atol=1e-13)


def test_not_causal_sees_all_and_positions_below_zero_see_nothing():
    K, V, table, rng = cache(2, 3, 1, 4, 16, 3)
    q = rng.standard_normal((11, 1, 16))
    o, lse, around = extend_paged(q, K, V, table, [3, 9], [1, 6, 10], 0.25)
    assert np.all(o[[0, 10]] == 0) and np.all(np.isneginf(lse[[0, 10]]))      # rows of no request
    assert np.all(o[1:3] == 0) and np.all(np.isneginf(lse[1:3]))              # 5 tokens, 3 cached: two before position 0
    np.testing.assert_allclose(o[3], V[table[0, 0], :, 0], atol=1e-15)        # position 0: its own value
    assert np.all(around >= np.abs(o) - 1e-15)
    all_, _, _ = extend_paged(q, K, V, table, [3, 9], [1, 6, 10], 0.25, causal=False)
    last, _, _ = extend_paged(q[5:6], K, V, table[:1], [3], [0, 1], 0.25)
    np.testing.assert_allclose(all_[5], last[0], atol=1e-15)                  # the last token sees all anyway
    np.testing.assert_allclose(all_[1:6].sum(), sum(extend_paged(q[i:i + 1], K, V, table[:1], [3], [0, 1], 0.25)[0].sum()
                                                    for i in range(1, 6)), atol=1e-13)


def test_rope_axes():
    assert fa.rope_axes((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert fa.rope_axes((2, 1, 3), in_turn=True) == bytes([0, 1, 2, 0, 2, 2])
    assert fa.rope_axes((4,)) == bytes(4) and fa.rope_axes((0, 2)) == bytes([1, 1])
    for bad in ((), (1, 1, 1, 1, 1), (0, 0), (3, -1)):
        with pytest.raises(ValueError):
            fa.rope_axes(bad)
