"""Chunk attention and rotations with several axes, run through both library
flavours by tests/test_gpu_debug_build_extend.py. Run as a script it writes the
results of the library selected by FA_DEBUG_LIBRARY to the file named on the
command line."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "tests")):
    if path not in sys.path:
        sys.path.insert(0, path)


def run_cases():
    """Results of every case as {name: CPU tensor}; asserts no device error."""
    import exact_tiled_attention_24_gb300 as fa
    from extend_cases import BF, extend_case, run
    g = torch.Generator().manual_seed(12)
    out = {}
    for i, (H, Hkv, d, bs, new, lens) in enumerate((
            (8, 2, 128, 16, [5, 1, 200, 0, 33], [300, 1, 200, 50, 160]), (4, 4, 64, 8, [130, 257, 3], [130, 700, 1000]),
            (8, 2, 128, 3, [5, 1, 90], [300, 1, 100]), (10, 2, 64, 5, [60, 7], [333, 90]),
            (130, 1, 64, 16, [3, 2], [260, 2]), (64, 64, 128, 16, [300, 2], [3000, 700]), (2, 1, 64, 128, [20, 4], [5, 0]))):
        q, caches, table, L, starts = extend_case(H, Hkv, d, bs, new, lens, seed=i, before=i % 2, after=i % 3, fill=0.0)
        total = caches[0].shape[0]
        codes = [t for _ in "kv" for t in (torch.randint(0, 256, (total, Hkv, bs, d // 2), generator=g).to(torch.uint8),
                                           torch.rand((total, Hkv, bs, d // 64, 2), generator=g).to(BF))]
        for kind, cache in (("bf16", caches), ("q4", codes)):
            for causal in (True, False):
                o, lse = run(fa, q, cache, table, L, starts, causal=causal)
                out[f"extend_{i}_{kind}_{causal}_o"], out[f"extend_{i}_{kind}_{causal}_lse"] = o.cpu(), lse.cpu()
    rn = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
    for sections, turn, inter in (((16, 24, 24), False, False), ((30, 2, 32), True, True)):
        axes = fa.rope_axes(sections, turn)
        cos, sin = fa.rope_tables(60, 128)
        pos = torch.randint(0, 60, (3, 2, 41), generator=g).to(torch.int32).cuda()
        q, k = rn(2, 5, 41, 128), rn(2, 2, 41, 128)
        kw = dict(positions=pos, axes=axes, q_weight=rn(128), k_weight=rn(128), interleaved=inter)
        for n, t in zip(("q", "k"), fa.qk_norm_rope(q, k, cos, sin, **kw)):
            out[f"axes_{turn}_{n}"] = t.cpu()
        for n, t in zip(("dq", "dk", "dqw", "dkw"), fa.qk_norm_rope_bwd(q, k, q, k, cos, sin, **kw)):
            out[f"axes_{turn}_{n}"] = t.cpu()
        cache = [torch.zeros((9, 2, 16, 128), dtype=BF, device="cuda") for _ in "kv"]
        table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
        t = torch.arange(41, dtype=torch.int32, device="cuda")
        qo = fa.append_paged(rn(41, 2, 128), rn(41, 2, 128), *cache, table, t, torch.zeros_like(t), cos, sin,
                             q=rn(41, 5, 128), rope_positions=pos[:, 0].contiguous(), axes=axes, interleaved=inter)
        out[f"axes_{turn}_append"], out[f"axes_{turn}_cache"] = qo.cpu(), cache[0].cpu()
    torch.cuda.synchronize()
    status = fa.last_device_error()
    assert status == 0, fa.FA_STATUS.get(status, status)
    return out


def main(path):
    import exact_tiled_attention_24_gb300 as fa
    assert fa.debug_checks() == (os.environ.get("FA_DEBUG_LIBRARY") == "1")
    torch.save(run_cases(), path)


if __name__ == "__main__":
    main(sys.argv[1])
