"""Decode over a 4-bit cache at the ends of the number range: queries so small
that 2^-e of their scale times the softmax scale is below fp32's normal range,
with keys as large as that; queries of zeros; large values.

Scores are a whole number times powers of two and the scale: the scale's own
rounding counts, 2^-20 where it is subnormal (20 bits of it are left at
2^-130), so a score is off by 2^-20 of itself, and lse by that and 2^-18."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import decode_paged, q4_unpack, q4_values
from test_gpu_decode_q4 import fa, q4_case, run  # noqa: F401

pytestmark = pytest.mark.gpu


def compare(q, cache, table, L, o, lse, scale):
    K, V = (q4_values(q4_unpack(cache[i].numpy()), np.nan_to_num(to_f64(cache[i + 1]))) for i in (0, 2))
    ref, rlse = decode_paged(to_f64(q), K, V, table.numpy(), L.numpy(), scale)
    top = 4 * np.abs(rlse).max() + 8      # scores of both signs
    assert np.abs(lse.double().cpu().numpy() - rlse).max() <= 2.0 ** -20 * top + 2.0 ** -18
    # o: its rounding, and e^(2 · a score's error) of every value
    assert np.abs(to_f64(o) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2 * (2.0 ** -20 * top + 2.0 ** -18) * np.abs(V).max()


@pytest.mark.parametrize("H,Hkv", [(2, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [-120, -122, -124, -125, -126])
def test_small_queries_against_large_keys(fa, d, e, H, Hkv):  # noqa: F811
    q, cache, table, L = q4_case(2, H, Hkv, d, 16, [200, 33], seed=-e + d)
    g = torch.Generator().manual_seed(d - e)
    one = torch.randint(0, d, (2, H, 1), generator=g)
    q = torch.zeros_like(q).scatter_(2, one, 2.0 ** e)
    live = ~cache[1].isnan().any(-1)
    cache[1][..., 0] = torch.where(live, 2.0 ** 124, float("nan"))   # keys up to 2^127: scores up to 2^(e + 127) scale
    cache[1][..., 1] = 0.0
    scale = 2.0 ** -(127 + e) * d ** -0.5 * 8 if e > -124 else d ** -0.5
    o, lse = run(fa, q, cache, table, L, 2, scale=scale)
    compare(q, cache, table, L, o, lse, scale)


@pytest.mark.parametrize("H,Hkv", [(2, 1), (8, 1)])
def test_queries_of_zeros(fa, H, Hkv):  # noqa: F811
    q, cache, table, L = q4_case(2, H, Hkv, 128, 16, [200, 33], seed=3)
    q[:] = 0
    o, lse = run(fa, q, cache, table, L, 2)
    compare(q, cache, table, L, o, lse, 128 ** -0.5)


@pytest.mark.parametrize("H,Hkv", [(2, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("power", [-100, 100])
def test_large_and_small_values(fa, H, Hkv, power):  # noqa: F811
    q, cache, table, L = q4_case(2, H, Hkv, 128, 16, [200, 33], seed=5)
    ref, rlse = run(fa, q, cache, table, L, 2)
    cache[3] *= 2.0 ** power
    o, lse = run(fa, q, cache, table, L, 2)
    assert torch.equal(o.double() * 2.0 ** -power, ref.double()) and torch.equal(lse, rlse)
