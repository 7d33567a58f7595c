"""Appends that make q_out themselves: the rows of padding and of skipped
tokens hold zeros, not what memory held."""
import pytest
import torch

from test_gpu_append_paged import Case, fa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("T,pad", [(40, 12), (700, 300)])
def test_rows_of_skipped_tokens_are_zeros(fa, q4, T, pad):  # noqa: F811
    s = Case(fa, T, 4, 6, 2, 128, 16, 128, True, seed=T, q4=q4, pad=pad)
    fn = fa.append_paged_q4 if q4 else fa.append_paged
    kw = s.kwargs()
    fn(s.k, s.v, *s.cache, s.table, s.pos, **kw)      # into a given q_out: rows stay 5.0
    given = kw.pop("q_out")
    live = torch.zeros(T, dtype=torch.bool)
    live[[t for t, _, _ in s.slots()]] = True
    assert int((~live).sum()) == pad and bool((given.cpu()[~live] == 5).all())
    for step in range(3):
        dirty = torch.full((T, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        del dirty                                      # the next tensor of its size may lie there
        if step == 2:
            s.table[:] = -1                            # no token has a block
            live[:] = False
        out = fn(s.k, s.v, *s.cache, s.table, s.pos, **kw)
        assert torch.equal(out.cpu()[live], given.cpu()[live]) and bool((out.cpu()[~live] == 0).all())
        assert fa.last_device_error() == (7 if step == 2 else 0)
