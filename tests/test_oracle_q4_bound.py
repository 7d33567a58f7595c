"""How far a value held in 4 bits may be off: max(s/2, 2^-8 (|z| + 8 s)). The
second is what the roundings of s and z to bf16 (8 significant bits: half a step
is up to 2^-8 of the number) shift the end levels by, and counts for groups far
from zero with a spread of a few bf16 steps."""
import numpy as np
import pytest

from oracle import q4_encode, q4_values
from oracle.cached import bf16


def groups_far_from_zero(rng, n, d=128):
    """bf16 rows around centres of 1 .. 2 (times powers of two), spread over a
    few bf16 steps."""
    centre = (1 + rng.random((n, d // 64, 1))) * 2.0 ** rng.integers(-30, 30, (n, d // 64, 1)) * rng.choice([-1, 1], (n, d // 64, 1))
    x = centre * (1 + 2.0 ** -7 * rng.integers(1, 9, (n, d // 64, 1)) * rng.random((n, d // 64, 64)))
    return bf16(x.reshape(n, d).astype(np.float32)).astype(np.float32)


def off(x):
    codes, pairs = q4_encode(x)
    s, z = (pairs[..., i].astype(np.float64).repeat(64, -1) for i in (0, 1))
    return np.abs(q4_values(codes, pairs) - x), s, np.abs(z)


def test_two_neighbouring_bf16_numbers():
    x = np.where(np.arange(64) % 2, np.float32(1.0078125), np.float32(1.0))[None]
    err, s, z = off(x)
    assert np.all(err <= np.maximum(s / 2, 2.0 ** -8 * (z + 8 * s)))
    assert err.max() > 1.5 * np.maximum(s / 2, 2.0 ** -9 * (z + 8 * s)).max()   # half of it does not hold


@pytest.mark.parametrize("seed", range(4))
def test_groups_far_from_zero(seed):
    err, s, z = off(groups_far_from_zero(np.random.default_rng(seed), 2000))
    bound = np.maximum(s / 2, 2.0 ** -8 * (z + 8 * s)) * (1 + 1e-5)
    assert np.all(err <= bound), (err / bound).max()
    assert (err > s / 2 * 1.1).any()          # the second term is what holds there
