"""Norms and rotation, appends and 4-bit decode steps, run through both library
flavours by tests/test_gpu_debug_build_cached.py. Run as a script it writes the
results of the library selected by FA_DEBUG_LIBRARY to the file named on the
command line."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def run_cases():
    """Results of every case as {name: CPU tensor}; asserts no device error."""
    import exact_tiled_attention_24_gb300 as fa
    BF, I32 = torch.bfloat16, torch.int32
    g = torch.Generator().manual_seed(11)
    rn = lambda *s: torch.randn(s, generator=g).to(BF).cuda()  # noqa: E731
    out = {}

    def keep(name, **tensors):
        torch.cuda.synchronize()
        status = fa.last_device_error()
        assert status == 0, f"{name}: device status {fa.FA_STATUS.get(status, status)}"
        out.update({f"{name}_{n}": t.cpu() for n, t in tensors.items()})

    for B, H, Hkv, N, d, rot, inter in ((2, 5, 2, 67, 128, 128, False), (1, 3, 3, 130, 64, 32, True),
                                        (3, 9, 1, 1, 128, 48, False)):
        qkv = rn(B, N, H + 2 * Hkv, d)
        q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
        cos, sin = fa.rope_tables(200, rot)
        pos = torch.randint(0, 200, (B, N), generator=g).to(I32).cuda()
        kw = dict(positions=pos, q_weight=rn(d), k_weight=rn(d), interleaved=inter)
        qo, ko = fa.qk_norm_rope(q, k, cos, sin, **kw)
        dq, dk, dqw, dkw = fa.qk_norm_rope_bwd(rn(B, H, N, d), rn(B, Hkv, N, d), q, k, cos, sin, **kw)
        keep(f"rope_{H}_{N}_{d}", q=qo, k=ko, dq=dq, dk=dk, dqw=dqw, dkw=dkw)
    for bs, d, H, Hkv in ((16, 128, 8, 2), (3, 128, 16, 1), (24, 64, 4, 4), (128, 64, 9, 1)):
        lens = [200, 1, 61]
        T = sum(lens)
        mb = 200 // bs + 1
        table = torch.randperm(3 * mb + 2, generator=g)[:3 * mb].view(3, mb).to(I32).cuda()
        req = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).to(I32).cuda()
        pos = torch.cat([torch.arange(n) for n in lens]).to(I32).cuda()
        cos, sin = fa.rope_tables(200, d)
        qkv = rn(T, H + 2 * Hkv, d)
        args = (qkv[:, H:H + Hkv], qkv[:, H + Hkv:])
        kw = dict(requests=req, cos=cos, sin=sin, q=qkv[:, :H], q_weight=rn(d), k_weight=rn(d))
        n = 3 * mb + 2
        dense = [torch.zeros((n, Hkv, bs, d), dtype=BF, device="cuda") for _ in "kv"]
        q4 = [torch.zeros(s, dtype=t, device="cuda") for _ in "kv"
              for s, t in (((n, Hkv, bs, d // 2), torch.uint8), ((n, Hkv, bs, d // 64, 2), BF))]
        held = [torch.zeros((T, Hkv, d), dtype=BF, device="cuda") for _ in "kv"]
        q1 = fa.append_paged(*args, *dense, table, pos, **kw)
        q2 = fa.append_paged_q4(*args, *q4, table, pos, k_values=held[0], v_values=held[1], **kw)
        keep(f"append_{bs}", q1=q1, q2=q2, kc=dense[0], vc=dense[1], kq=q4[0], ks=q4[1], vq=q4[2], vs=q4[3], kh=held[0])
        L = torch.tensor(lens, dtype=I32).cuda()
        last = torch.tensor([199, 200, 261], device="cuda")
        for S in (1, 3):
            o, lse = fa.decode_paged_q4(q2[last], *q4, table, L, n_splits=S)
            keep(f"decode_q4_{bs}_{S}", o=o, lse=lse)
    return out


def main(path):
    import exact_tiled_attention_24_gb300 as fa
    assert fa.debug_checks() == (os.environ.get("FA_DEBUG_LIBRARY") == "1")
    torch.save(run_cases(), path)


if __name__ == "__main__":
    main(sys.argv[1])
