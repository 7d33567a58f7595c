"""extend_paged_q4 over steps below the smallest normal number: codes are read
back as z + s (n - 8), rounded once, for any s."""
import numpy as np
import pytest
import torch

from extend_cases import BF, run
from oracle import q4_pack, q4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


@pytest.mark.parametrize("d", [64, 128])
def test_steps_of_any_size(fa, d):
    """One key a request, weight 1: o is the value read back. Steps are 1 to 255
    times 2^-133 (bf16's smallest number), centres large enough for the results
    to be normal."""
    n = 255
    g = torch.Generator().manual_seed(2)
    codes = torch.arange(16).repeat(n * d // 16).view(n, 1, 1, d)
    codes = codes[..., torch.randperm(d, generator=g)]
    s = torch.arange(1, n + 1).double()[:, None] * 2.0 ** -133
    z = (1 + torch.rand((n, d // 64), generator=g).double()) * 2.0 ** torch.randint(-121, -117, (n, d // 64), generator=g)
    pairs = torch.stack([s.expand(n, d // 64).to(torch.float32).to(BF), z.to(torch.float32).to(BF)], -1).view(n, 1, 1, d // 64, 2)
    assert bool((pairs[..., 0].double()[:, 0, 0] == s).all())
    packed = torch.from_numpy(q4_pack(codes.numpy()))
    ref = q4_values(codes.numpy(), pairs.double().numpy())  # exact in 64 bits
    step = 2.0 ** (np.floor(np.log2(np.abs(ref))) - 7)
    assert step.min() >= 2.0 ** -133
    want = torch.from_numpy(np.rint(ref / step) * step).to(torch.float32)
    table = torch.arange(n, dtype=torch.int32)[:, None].contiguous()
    zero = torch.zeros_like(packed), torch.zeros_like(pairs)
    q = torch.zeros((n, 1, d), dtype=BF)
    o, _ = run(fa, q, (*zero, packed, pairs), table, torch.ones(n, dtype=torch.int32), torch.arange(n + 1, dtype=torch.int32))
    assert torch.equal(o[:, 0].float().cpu(), want[:, 0, 0])
