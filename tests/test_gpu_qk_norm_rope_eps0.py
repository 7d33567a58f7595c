"""The gradient of norms and rotation with eps = 0, where a row of zeros has no
finite 1 / rms: rows that only fill up a tile of the kernel must not count, nor
tokens whose position lies outside the tables, whatever they hold. Bounds as in
test_gpu_qk_norm_rope.py."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_24_gb300.workloads import to_f64
from oracle import norm_rope_bwd
from test_gpu_qk_norm_rope import case, f64, fa, rows_max  # noqa: F401

pytestmark = pytest.mark.gpu


def output_gradients(q, k, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda() for x in (q, k)]


@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,N", [(1, 1), (1, 17), (1, 33), (3, 11), (2, 32)])
def test_weight_gradients_without_eps(fa, B, N, d, rot):  # noqa: F811
    q, k, cos, sin, pos, qw, kw = case(B, 3, 2, N, d, rot, "packed", torch.bfloat16, "own" if rot else None, seed=N + d)
    dqo, dko = output_gradients(q, k, N)
    grads = fa.qk_norm_rope_bwd(dqo, dko, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, eps=0.0)
    assert fa.last_device_error() == 0
    P = None if pos is None else pos.cpu().numpy()
    for dy, x, w, dx, dw in ((dqo, q, qw, grads[0], grads[2]), (dko, k, kw, grads[1], grads[3])):
        args = (f64(cos), f64(sin), P, 0.0)
        rdx, rdw = norm_rope_bwd(to_f64(dy), to_f64(x), f64(w), *args)
        back, _ = norm_rope_bwd(to_f64(dy), to_f64(x), None, *args)
        r = 1 / np.sqrt(np.mean(to_f64(x) ** 2, -1, keepdims=True))
        h, n = back * f64(w), to_f64(x) * r
        rows = B * N * x.shape[1]
        turned = 2.0 ** -21 * (rows_max(to_f64(dy)) * np.abs(n)).sum(axis=(0, 1, 2))
        assert np.all(np.abs(f64(dw) - rdw) <= (rows + 64) * 2.0 ** -24 * np.abs(back * n).sum(axis=(0, 1, 2)) + turned)
        scale = rows_max(r * h) + rows_max(r * n) * np.abs(np.mean(h * n, -1, keepdims=True))
        assert np.all(np.abs(to_f64(dx) - rdx) <= 2.0 ** -8 * np.abs(rdx) + 2.0 ** -17 * scale)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_without_a_position_add_nothing(fa, d, eps):  # noqa: F811
    q, k, cos, sin, pos, qw, kw = case(1, 2, 1, 40, d, 64, "plain", torch.float32, "own", seed=9)
    dqo, dko = output_gradients(q, k, 3)
    bad = {3: 0.0, 7: float("nan"), 39: float("inf")}
    for t, fill in bad.items():
        q[:, :, t], k[:, :, t], dqo[:, :, t] = fill, fill, float("nan")
        pos[0, t] = -1 if t == 3 else cos.shape[0] + t
    dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(dqo, dko, q, k, cos, sin, positions=pos, q_weight=qw, k_weight=kw, eps=eps)
    assert fa.last_device_error() == 7 and fa.last_device_error() == 0
    good = [t for t in range(40) if t not in bad]
    ok = [x[:, :, good].contiguous() for x in (dqo, dko, q, k)]
    ref = fa.qk_norm_rope_bwd(*ok, cos, sin, positions=pos[:, good].contiguous(), q_weight=qw, k_weight=kw, eps=eps)
    assert fa.last_device_error() == 0
    for x, y in zip((dq, dk), ref[:2]):
        assert torch.equal(x[:, :, good], y) and bool((x[:, :, list(bad)] == 0).all())
    # the same terms in another order: 40 rows of 3 heads at most, 2^-24 of a
    # term's size each
    for x, y in zip((dqw, dkw), ref[2:]):
        assert bool(y.isfinite().all())
        assert float((x - y).abs().max()) <= 2 * 40 * 2 * 2.0 ** -24 * float(40 * 2 * max(t.float().abs().max() for t in ok[:2]) * d ** 0.5)
