"""How a chunk call's work is cut (fa_extend_plan.cuh), on the host: the
functions that the kernel and the merge evaluate, against an enumeration of all
items and key tiles (tests/extend_plan_host.cu has the checks)."""
import ctypes
import os
import random
import subprocess

import pytest

from exact_tiled_attention_24_gb300 import build as fabuild

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    lib = fabuild.build()
    out = str(tmp_path_factory.mktemp("plan") / "plan_host.so")
    cmd = [fabuild._nvcc(), *fabuild.ARCH, "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-I", fabuild.CSRC, "-I",
           os.path.join(fabuild.ROOT, "include"), "-shared", "-o", out, os.path.join(TESTS, "extend_plan_host.cu"), lib,
           "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    L = ctypes.CDLL(out)

    def check(T, H, Hkv, d, bs, max_blocks, starts, lens, causal=True, q4=False):
        """(chunks of the most cut request, long items, largest slot, requests taken for empty, keys a chunk)"""
        B = len(lens)
        assert len(starts) == B + 1
        got = (ctypes.c_int * 5)()
        line = L.plan_check(T, B, H, Hkv, d, bs, max_blocks, int(causal), int(q4), (ctypes.c_int * (B + 1))(*starts),
                            (ctypes.c_int * B)(*lens), got)
        assert line == 0, (f"extend_plan_host.cu:{line}", T, H, Hkv, d, bs, max_blocks, starts, lens, causal, q4)
        return list(got)

    return check


def starts_of(new, first=0):
    out = [first]
    for n in new:
        out.append(out[-1] + n)
    return out


def blocks_for(longest, bs):
    return max(1, -(-longest // bs))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv,d,new,lens,bf16,codes", [
    (256, 4, 128, [80], [220000], 2, 2),
    (256, 4, 128, [66], [220000], 3, 3),   # 2.2 shares
    (256, 4, 128, [56], [220000], 3, 1),   # 2.7
    (16, 16, 64, [1500, 3, 1300], [200000, 9, 100000], 2, 2),
    (16, 4, 64, [3500], [200000], 1, 1),   # 2.7
    (6, 6, 128, [5, 2600, 2], [17, 150000, 800], 3, 3),
    (256, 4, 128, [36], [220000], 5, 1),   # 4.2
    (256, 4, 128, [32], [220000], 1, 1),   # 4.75
    (16, 4, 128, [350], [300000], 1, 1),   # 6.3
    (16, 2, 128, [160], [300000], 1, 1),   # five items a head
    (16, 2, 128, [200], [300000], 1, 1),   # over codes three pieces of L2's size, but eleven shares
])
def test_chunked(plan, H, Hkv, d, new, lens, bf16, codes, causal, q4):
    """Requests that are cut into chunks of keys, alone and among others."""
    chunks = codes if q4 else bf16
    got = plan(sum(new), H, Hkv, d, 16, blocks_for(max(lens), 16), starts_of(new), lens, causal, q4)
    assert got[0] == chunks and (got[1] > 0) == (chunks > 1), got


def test_random_calls(plan):
    """Ordinary calls, some of lengths that are cut into chunks."""
    rng = random.Random(5)
    cut = 0
    for _ in range(2200):
        B = rng.choice([1, 1, 2, 3, 5, 9, 40])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 5, 16, 64, 130])
        d, bs = rng.choice([64, 128]), rng.choice([1, 3, 16, 64, 200])
        tpt = max(1, 128 // (H // Hkv))
        new = [rng.choice([0, 1, rng.randint(0, 40 * tpt)]) for _ in range(B)]
        most = rng.choice([300, 5000, 400000])
        lens = [max(0, n + rng.randint(-3, most)) for n in new]
        before, after = rng.choice([0, 0, 7]), rng.choice([0, 0, 50])
        got = plan(max(1, before + sum(new) + after), H, Hkv, d, bs, blocks_for(max(lens), bs) + rng.choice([0, 5]),
                   starts_of(new, before), lens, rng.random() < 0.7, rng.random() < 0.5)
        assert got[3] == 0
        cut += got[0] > 1
    assert cut > 100


@pytest.mark.parametrize("q4", [False, True])
def test_starts_that_go_down_and_up_again(plan, q4):
    """Requests that cover rows twice: more slots and long items than the host
    made room for, if they were all taken."""
    got = plan(400, 32, 8, 128, 16, 1024, [0, 400, 0, 400], [16384] * 3, True, q4)
    assert got[3] == 2
    got = plan(1281, 4, 4, 128, 16, 3840, [0, 1281, 0, 1281], [61440] * 3, True, q4)
    assert got[3] == 2
    # an overlap by one row, starts in order again behind it; a request of no rows is behind anything
    assert plan(40, 8, 2, 128, 16, 4, [0, 10, 9, 20, 20, 40], [60] * 5)[3] == 2
    assert plan(40, 8, 2, 128, 16, 4, [0, 10, 10, 5, 5, 40], [60] * 5)[3] == 2
    # numbers out of range hold up none of the others
    assert plan(38, 8, 2, 128, 16, 4, [-1, 5, 35, 38], [60] * 3)[3] == 1
    assert plan(38, 8, 2, 128, 16, 4, [0, 2 ** 31 - 1, 5, 38], [60] * 3)[3] == 2


def test_random_starts(plan):
    rng = random.Random(6)
    dropped = 0
    for _ in range(600):
        B, Hkv = rng.choice([1, 2, 3, 6, 30]), rng.choice([1, 2, 8])
        H = Hkv * rng.choice([1, 4, 64])
        T = rng.choice([1, 50, 900])
        some = [0, T, -1, T + 1, 2 ** 31 - 1, -2 ** 31]
        starts = [rng.choice(some) if rng.random() < 0.4 else rng.randint(0, T) for _ in range(B + 1)]
        if rng.random() < 0.4:
            starts = sorted(starts)
        lens = [rng.choice([0, 1, 100, 2 ** 31 - 1, -5, rng.randint(0, 200000)]) for _ in range(B)]
        dropped += plan(T, H, Hkv, 128, 16, 12500, starts, lens, rng.random() < 0.7, rng.random() < 0.5)[3]
    assert dropped > 500


def test_workspace_is_what_the_parts_need(plan):
    """Two parts a CTA, and as many again for long items at most."""
    import exact_tiled_attention_24_gb300 as fa
    part = 256 * 129 * 4 + 24
    assert fa.extend_workspace_bytes(1 << 17, 1, 32, 8, 128, 16, 1 << 13) <= 4 * 152 * part
    assert fa.extend_workspace_bytes(1 << 17, 1, 1, 1, 128, 16, 1 << 13) <= 4 * 152 * part
    assert fa.extend_workspace_bytes(350, 1, 16, 4, 128, 16, 1 << 13) <= 4 * 152 * part


def test_the_gpu_tests_cases(plan):
    """The calls of test_gpu_extend_chunks.py are cut as they say."""
    from extend_chunk_cases import CASES
    for kind, H, Hkv, d, bs, new, lens, want in CASES.values():
        for causal in (True, False):
            got = plan(sum(new), H, Hkv, d, bs, blocks_for(max(lens), bs), starts_of(new), lens, causal, kind == "q4")
            assert got[0] == max(want) and got[1] > 0
