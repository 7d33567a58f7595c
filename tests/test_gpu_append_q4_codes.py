"""4-bit codes of keys that are normed but not rotated: the definition rounds
the product with the weight and the difference from the centre each by itself,
so the codes are those of the same operations on the host, bit for bit.

The norm's own arithmetic is made exact: magnitudes 1, 3, 5, 7 with a mean
square of 16 and eps = 0 give r = 1/4, and x r is exact. The weights bring every
product near one value v, so the steps are about 2^-12 v: then a code moves
whenever the difference is formed from the unrounded product, once in some
2^14 values."""
import numpy as np
import pytest
import torch

from oracle import q4_encode, q4_pack
from test_gpu_append_paged import fa  # noqa: F401

pytestmark = pytest.mark.gpu
CALLS = 1500


def magnitudes(d, rng):
    """d numbers of 1, 3, 5, 7 whose mean square is 16: per 64, 24 + 15 + 15 + 10."""
    x = np.concatenate([np.repeat([1.0, 3.0, 5.0, 7.0], [24, 15, 15, 10]) for _ in range(d // 64)])
    assert (x * x).mean() == 16
    return rng.permutation(x)


@pytest.mark.parametrize("d,rot", [(64, 0), (128, 0), (128, 64), (64, 16)])
def test_codes_of_normed_keys(fa, d, rot):  # noqa: F811
    rng = np.random.default_rng(d + rot)
    dev = "cuda"
    cache = [t for _ in "kv" for t in (torch.zeros((1, 1, CALLS, d // 2), dtype=torch.uint8, device=dev),
                                       torch.zeros((1, 1, CALLS, d // 64, 2), dtype=torch.bfloat16, device=dev))]
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    # turning by no angle: products with 1 and 0 are exact too
    cos, sin = (f((CALLS, rot // 2), device=dev) for f in (torch.ones, torch.zeros)) if rot else (None, None)
    want = np.empty((CALLS, d), dtype=np.float32)
    for i in range(CALLS):
        x = magnitudes(d, rng).astype(np.float32)
        v = np.float32(1.0) + rng.random(dtype=np.float32)
        w = (v * (1 + 2.0 ** -10 * rng.standard_normal(d)) / (x / 4)).astype(np.float32)
        want[i] = x * np.float32(0.25) * w
        k = torch.from_numpy(x).to(torch.bfloat16).to(dev)[None, None]
        fa.append_paged_q4(k, k, *cache, table, torch.tensor([i], dtype=torch.int32, device=dev), cos=cos, sin=sin,
                           k_weight=torch.from_numpy(w).to(dev), eps=0.0)
    assert fa.last_device_error() == 0
    codes, pairs = q4_encode(want)
    np.testing.assert_array_equal(cache[1][0, 0].float().cpu().numpy(), pairs)
    np.testing.assert_array_equal(cache[0][0, 0].cpu().numpy(), q4_pack(codes))


def test_values_far_from_zero_are_within_the_bound(fa):  # noqa: F811
    from oracle import q4_unpack, q4_values
    from test_oracle_q4_bound import groups_far_from_zero
    T = 400
    x = groups_far_from_zero(np.random.default_rng(9), T)
    v = torch.from_numpy(x).to(torch.bfloat16).cuda()[:, None]
    cache = [t for _ in "kv" for t in (torch.zeros((1, 1, T, 64), dtype=torch.uint8, device="cuda"),
                                       torch.zeros((1, 1, T, 2, 2), dtype=torch.bfloat16, device="cuda"))]
    at = torch.arange(T, dtype=torch.int32, device="cuda")
    fa.append_paged_q4(v, v, *cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), at, torch.zeros_like(at))
    assert fa.last_device_error() == 0
    codes, pairs = q4_encode(x)
    for c, p in (cache[:2], cache[2:]):
        np.testing.assert_array_equal(c[0, 0].cpu().numpy(), q4_pack(codes))
        got = p[0, 0].double().cpu().numpy()
        np.testing.assert_array_equal(got, pairs.astype(np.float64))
        s, z = (got[..., i].repeat(64, -1) for i in (0, 1))
        held = q4_values(q4_unpack(c[0, 0].cpu().numpy()), got)
        assert np.all(np.abs(held - x) <= np.maximum(s / 2, 2.0 ** -8 * (np.abs(z) + 8 * s)) * (1 + 1e-5))
