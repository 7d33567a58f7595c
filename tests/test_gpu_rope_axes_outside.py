"""Gradients of rotations with several axes where a token's position on one axis
is outside the tables: that token has no gradient and adds nothing to the
weights', whatever its rows hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("d,sections", [(128, (16, 24, 24)), (64, (3, 9, 4)), (128, (0, 40, 24))])
def test_gradient(fa, d, sections, inter, norm):
    B, H, Hkv, N, n_pos = 2, 5, 2, 37, 40
    g = torch.Generator().manual_seed(d + sum(sections))
    rn = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
    axes = fa.rope_axes(sections, in_turn=inter)
    cos, sin = fa.rope_tables(n_pos, 2 * len(axes))
    pos = torch.randint(0, n_pos, (3, B, N), generator=g).to(I32).cuda()
    q, k, dq, dk = rn(B, H, N, d), rn(B, Hkv, N, d), rn(B, H, N, d), rn(B, Hkv, N, d)
    kw = dict(axes=axes, interleaved=inter, eps=0.0)
    if norm:
        kw |= dict(q_weight=rn(d), k_weight=rn(d))
    gone = torch.zeros((B, N), dtype=torch.bool, device="cuda")
    for axis, b, n, x in ((0, 0, 0, -1), (1, 0, 20, n_pos), (2, 1, 36, 2 ** 31 - 1), (1, 1, 7, -2 ** 31)):
        gone[b, n] = True
        pos[axis, b, n] = x
    # the same gradients from tokens that are all in the tables and those ones' output gradients 0
    inside = torch.where((pos >= 0) & (pos < n_pos), pos, 0)
    rows = gone[:, None, :, None]
    ref = fa.qk_norm_rope_bwd(dq.masked_fill(rows, 0), dk.masked_fill(rows, 0), q, k, cos, sin, positions=inside, **kw)
    assert fa.last_device_error() == 0
    # rows that nothing may read into a sum: NaN, and zeros (no finite 1/rms at eps = 0)
    for fill in (float("nan"), 0.0):
        args = [t.masked_fill(rows, fill) for t in (dq, dk, q, k)]
        got = fa.qk_norm_rope_bwd(*args, cos, sin, positions=pos, **kw)
        torch.cuda.synchronize()
        assert fa.last_device_error() == 7
        for a, b in zip(got[:2], ref[:2]):
            assert bool((a.masked_select(rows.expand_as(a)) == 0).all())
            assert torch.equal(a.masked_fill(rows, 0), b.masked_fill(rows, 0))
        for a, b in zip(got[2:], ref[2:]):
            assert (a is None and b is None) or torch.equal(a, b)
