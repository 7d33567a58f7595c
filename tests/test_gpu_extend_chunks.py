"""extend_paged and extend_paged_q4 where the keys of a request are cut into
two to five chunks: every load path, with other requests before and after,
all keys and causal, captured and replayed with lengths that are cut and that
are not, and on the bounds-checked build."""
import os
import subprocess
import sys

import pytest
import torch

from extend_chunk_cases import CASES, TILE, attention64, chunks, inputs, run

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = sorted(CASES)


@pytest.fixture(scope="module")
def fa():
    from exact_tiled_attention_24_gb300 import build
    build.build()
    import exact_tiled_attention_24_gb300 as m
    return m


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_the_cases_are_cut(name, causal):
    kind, H, Hkv, d, bs, new, lens, want = CASES[name]
    assert chunks(kind, H, Hkv, d, bs, new, lens, causal, -(-max(lens) // bs)) == want and max(want) >= 2


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_every_key_is_counted_once(fa, name, causal):
    """q = 0: each weight is 1 and each sum a whole number below 2^24, both
    exact; the normalised parts, their weights e^(lse - lse') (lse within
    2^-19.5) and the sums over 32 parts at most cost under 2^-16 of o, its
    rounding 2^-8. lse: as in extend_cases.check, with scores that are exact."""
    q, caches, table, lens, starts = inputs(name, 3, counting=True)
    o, lse = run(fa, q, caches, table, lens, starts, causal=causal)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    d = q.shape[2]
    for b, length in enumerate(lens.tolist()):
        lo, hi = starts[b].item(), starts[b + 1].item()
        for t in range(lo, hi):
            seen = length - (hi - lo) + (t - lo) + 1 if causal else length
            tiles = torch.full((-(-seen // TILE),), float(TILE), dtype=torch.float64, device="cuda")
            tiles[-1] = seen - TILE * (len(tiles) - 1)
            want = torch.zeros(d, dtype=torch.float64, device="cuda")
            want.index_add_(0, torch.arange(len(tiles), device="cuda") % d, tiles)
            want /= seen
            err = (o[t].double() - want).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -16) * want).all()), (b, t)
            log = torch.tensor(float(seen), dtype=torch.float64).log().item()
            assert bool(((lse[t].double() - log).abs() <= 2.0 ** -20 * (log + 1)).all()), (b, t)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_against_64_bits(fa, name, causal):
    """Peaked scores; the bounds of extend_cases.check."""
    args = inputs(name, 11)
    o, lse = run(fa, *args, causal=causal)
    torch.cuda.synchronize()
    assert fa.last_device_error() == 0
    ro, rl, around, reach = attention64(*args, causal)
    e = 2.0 ** -16 * reach
    tol = (2.0 ** -8 * (around + ro.abs()) + 2 * e[..., None] * around) * 1.01
    assert bool(((o.double() - ro).abs() <= tol).all())
    assert bool(((lse.double() - rl).abs() <= e + 2.0 ** -20 * (rl.abs() + 1)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["boxes", "gathered", "codes"])
def test_a_captured_call_is_cut_or_not_as_its_lengths_say(fa, name):
    kind, H, Hkv, d, bs, new, lens, most = CASES[name]
    args = inputs(name, 5)
    q, caches, table, L, starts = args
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    run(fa, *args, out=o, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(fa, *args, out=o, lse=lse)
    cut = set()
    for length, n in ((lens[0], new[0]), (700, new[0]), (lens[0] // 2 + 77, new[0] - 1), (lens[0], 2), (lens[0] - 1, new[0])):
        L.fill_(length)
        starts[1:].fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        ro, rl = torch.empty_like(o), torch.empty_like(lse)
        run(fa, *args, out=ro, lse=rl)
        torch.cuda.synchronize()
        assert torch.equal(o[:n], ro[:n]) and torch.equal(lse[:n], rl[:n])
        cut.add(chunks(kind, H, Hkv, d, bs, [n], [length], True, table.shape[1])[0])
    assert fa.last_device_error() == 0
    assert cut == set(range(1, most[0] + 1))


@pytest.mark.gpu
def test_the_debug_build_agrees(fa, tmp_path):
    """No bounds check fires and the results are the release build's bit for bit."""
    from exact_tiled_attention_24_gb300 import build
    build.build(debug=True)
    path = tmp_path / "debug.pt"
    r = subprocess.run([sys.executable, os.path.join(HERE, "extend_chunk_cases.py"), str(path)],
                       env=dict(os.environ, FA_DEBUG_LIBRARY="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    debug = torch.load(path)
    for name in CASES:
        for causal in (True, False):
            o, lse = run(fa, *inputs(name, 7), causal=causal)
            assert torch.equal(o.cpu(), debug[f"{name} {causal} o"]), name
            assert torch.equal(lse.cpu(), debug[f"{name} {causal} lse"]), name
