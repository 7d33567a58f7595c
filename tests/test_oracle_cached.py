"""The fp64 definitions of norms, rotation and 4-bit codes, against what they
have to satisfy."""
import numpy as np
import pytest

from oracle import append_slots, norm_rope, norm_rope_bwd, q4_encode, q4_pack, q4_unpack, q4_values


def tables(n_pos, rot):
    angle = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_scores_a_function_of_distance(interleaved):
    # q at position a, k at position b: their product depends on a - b alone
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    cos, sin = tables(200, 64)
    at = lambda x, p: norm_rope(x, None, cos, sin, [p], interleaved=interleaved)  # noqa: E731
    s = [float((at(q, a) * at(k, a - 30)).sum()) for a in (30, 77, 199)]
    np.testing.assert_allclose(s, s[0], rtol=1e-12)
    np.testing.assert_allclose((at(q, 50) ** 2).sum(), (q ** 2).sum(), rtol=1e-12)


def test_norm_gives_unit_mean_square_times_weight():
    x = np.random.default_rng(2).standard_normal((2, 3, 4, 64)) * 7
    w = np.linspace(0.5, 2, 64)
    y = norm_rope(x, w, eps=0.0)
    np.testing.assert_allclose(((y / w) ** 2).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("interleaved,rot", [(False, 64), (True, 32)])
def test_gradient_matches_differences(interleaved, rot):
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((2, 2, 3, 64)), rng.standard_normal((2, 2, 3, 64)), rng.standard_normal(64)
    cos, sin = tables(10, rot)
    pos = [[4, 0, 9], [1, 2, 3]]
    f = lambda x_, w_: float((norm_rope(x_, w_, cos, sin, pos, 1e-3, interleaved) * dy).sum())  # noqa: E731
    dx, dw = norm_rope_bwd(dy, x, w, cos, sin, pos, 1e-3, interleaved)
    for _ in range(20):
        u = rng.standard_normal(x.shape)
        num = (f(x + 1e-5 * u, w) - f(x - 1e-5 * u, w)) / 2e-5
        np.testing.assert_allclose((dx * u).sum(), num, rtol=1e-6, atol=1e-7)
        u = rng.standard_normal(64)
        num = (f(x, w + 1e-5 * u) - f(x, w - 1e-5 * u)) / 2e-5
        np.testing.assert_allclose((dw * u).sum(), num, rtol=1e-6, atol=1e-7)


def test_codes_round_trip_and_bound():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((50, 128)) * 10.0 ** rng.integers(-20, 20, (50, 1))
         + rng.integers(-3, 4, (50, 1))).astype(np.float32)
    codes, pairs = q4_encode(x)
    assert codes.max() == 15 and codes.min() == 0
    np.testing.assert_array_equal(q4_unpack(q4_pack(codes)), codes)
    s, z = pairs[..., 0].repeat(64, -1), pairs[..., 1].repeat(64, -1)
    bound = np.maximum(s / 2, 2.0 ** -9 * (np.abs(z) + 8 * s)) * (1 + 1e-5) + 1e-42
    assert np.all(np.abs(q4_values(codes, pairs) - x) <= bound)


def test_codes_of_constant_and_non_finite_groups():
    x = np.zeros((4, 128), dtype=np.float32)
    x[0] = 1.5
    x[1, 3], x[2, 70], x[3, 0] = np.nan, np.inf, -np.inf
    codes, pairs = q4_encode(x)
    v = q4_values(codes, pairs)
    assert np.all(v[0] == 1.5) and np.all(codes[0] == 8)
    assert np.all(np.isnan(v[1, :64])) and np.all(v[1, 64:] == 0)
    assert np.all(np.isnan(v[2, 64:])) and np.all(v[2, :64] == 0)
    assert np.all(np.isnan(v[3, :64]))


def test_append_slots_skip_padding():
    table = np.array([[5, 2], [7, 1]])
    assert append_slots(table, [0, 9, -1, 3], [1, 0, 0, -1], 8) == [(0, 7, 0), (1, 2, 1)]
    assert append_slots(table, [8, 1], None, 8) == [(0, 2, 0), (1, 7, 1)]
