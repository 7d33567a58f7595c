"""What decode over a 4-bit cache loses beside the rounding of its result.

Scores are made exact, so that only the output's own arithmetic is left: a
query has one element that is not 0, a power of two, and every key the step
1/4 and the centre 0, so a score is q (n - 8) / 4 times the scale, a whole
number times the scale. Bounds, with S = Σ p |s (n - 8)| and Z = Σ p |z| over
a request's keys (Σ p = 1):

* the result's rounding to bf16: half of the step at its magnitude;
* p s as two bf16 numbers, 2^-8 each: 2^-16 S;
* p from a score: the scale, its product with the score and the subtraction of
  the reference, 2^-24 each of at most 16 in log2 units, then the exponential
  (2^-22): under 2^-17 of p, in the numerator and in Σ p: 2^-16 (S + Z);
* sums in fp32, cut off at 2^-23 of what they hold. The codes' offsets are in
  them until they cancel: 31 Σ p s over up to 16 keys of a warp, with p at most
  8 times its mean, so 31 · 16 · 8 times the mean of p s, cut off once every 16
  keys: under keys / 16 · 2^12 · 2^-23 of it, where S is about 4 · keys of it
  (|n - 8| is 4 on average): 2^-17 S. The centres and Σ p: fewer than 2^8
  additions of 2^-24: 2^-16 Z.

Together under 2^-14 (S + Z). One bf16 number for p s is off by up to 2^-8 of
each key's part, which no such bound holds. lse is off as Σ p is, 2^-17, and by
its logarithm and rounding, 2^-20 of it."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import decode_paged, q4_unpack, q4_values
from test_gpu_decode_q4 import fa, q4_case, run  # noqa: F401

pytestmark = pytest.mark.gpu
SCALE = 0.25


def half_step(x):
    """Half of bf16's step at each magnitude (8 significant bits)."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def exact_scores(B, H, Hkv, d, bs, lens, seed):
    q, cache, table, L = q4_case(B, H, Hkv, d, bs, lens, seed)
    g = torch.Generator().manual_seed(seed)
    one = torch.randint(0, d, (B, H, 1), generator=g)
    q = torch.zeros_like(q).scatter_(2, one, torch.where(torch.rand(B, H, 1, generator=g) < 0.5, 4.0, -8.0).to(q.dtype))
    cache[1][..., 0], cache[1][..., 1] = 0.25, 0.0
    return q, cache, table, L


CASES = [
    # B, H, Hkv, d, bs, lens, n_splits
    (2, 1, 1, 64, 16, [40, 200], 1),
    (2, 8, 2, 128, 16, [64, 200], 1),      # 4 query heads a K/V head
    (3, 6, 2, 128, 3, [31, 150, 77], 2),   # 3, gathered
    (2, 5, 1, 64, 16, [64, 130], 2),       # 5
    (2, 16, 2, 128, 16, [50, 200], 1),     # 8
    (2, 8, 1, 128, 1, [50, 200], 2),
    (2, 16, 1, 128, 16, [64, 200], 1),     # 16
    (1, 18, 1, 64, 7, [150], 2),           # 16 + 2
]


@pytest.mark.parametrize("c", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_output_is_off_by_its_own_rounding(fa, c):  # noqa: F811
    B, H, Hkv, d, bs, lens, S = c
    q, cache, table, L = exact_scores(B, H, Hkv, d, bs, lens, seed=sum(lens) + H)
    o, lse = run(fa, q, cache, table, L, S, scale=SCALE)
    Q, kp, vp = to_f64(q), np.nan_to_num(to_f64(cache[1])), np.nan_to_num(to_f64(cache[3]))
    K, vn = q4_values(q4_unpack(cache[0].numpy()), kp), q4_unpack(cache[2].numpy())
    ref, rlse = decode_paged(Q, K, q4_values(vn, vp), table.numpy(), L.numpy(), SCALE)
    zero = np.zeros_like(vp[..., 0])
    spread, _ = decode_paged(Q, K, np.abs(q4_values(vn, np.stack([vp[..., 0], zero], -1))), table.numpy(), L.numpy(), SCALE)
    centre, _ = decode_paged(Q, K, np.abs(q4_values(vn, np.stack([zero, vp[..., 1]], -1))), table.numpy(), L.numpy(), SCALE)
    err = np.abs(to_f64(o) - ref)
    bound = half_step(np.maximum(np.abs(ref), np.abs(to_f64(o)))) + 2.0 ** -14 * (spread + centre)
    assert np.all(err <= bound), (int((err > bound).sum()), float((err - bound).max()))
    assert np.abs(lse.double().cpu().numpy() - rlse).max() <= 2.0 ** -17 + 2.0 ** -20 * np.abs(rlse).max()
