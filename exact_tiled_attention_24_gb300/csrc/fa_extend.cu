// Attention of chunks of new tokens over a paged KV cache, in bf16 or in
// 4-bit codes: a packed, ragged batch of any requests' tokens (whole prompts,
// parts of prompts, a few tokens to be verified, single tokens).
//
//   o_i = Σ_j softmax_j(scale q_i·k_j) v_j,  lse_i = ln Σ_j e^(scale q_i·k_j)
//
// over the keys j that token i sees: those up to its own position (causal),
// or all of its request's. Tile by tile with a running maximum and sum, as in
// the forward (fa_fwd.cu), whose two tensor-core products, order of products
// and threshold for rescaling are used here too.
//
// A query tile holds up to 128 rows: tpt tokens with the `heads` query heads
// that share a K/V head (row = token · heads + head), so a K/V tile is read
// once for all of them. A CTA works on items of two query tiles, a share of
// all (item, key tile) units of the call (fa_extend_plan.cuh), one piece (the
// part of an item in its share) after another without a pause: while the last
// products of a piece run, the next one's keys are on their way.
//
// Roles:
//   warp 0       the pieces of the CTA's share, into a ring of descriptors
//   warp 1       TMEM owner and MMA issuer (warp-uniform, one elected lane)
//   warp 2       K and V tiles as TMA boxes (block sizes that are a multiple of
//                8 dividing 128), one box per cache block
//   warp 3       Q tiles
//   warps 4..7   softmax of the first query tile, one thread per row
//   warps 8..11  softmax of the second
//   warps 12..15 (other block sizes, 4-bit caches) K and V tiles: gathered row
//                by row, or codes unpacked to bf16 into the products' layout
// TMEM columns: S0 0.., S1 128.., O0 256.., O1 384... P overwrites S.
//
// What bounds it (32 + 8 heads, d = 128, 2070 MHz): with full tiles the tensor
// pipe, as in the forward: 2048 clocks of products in 3300 a unit (a prompt of
// 8192 tokens 409 to 419 us, 1024 tokens at 131072 keys 1.45 to 1.49 ms, 1470 to
// 1510 TFLOP/s). With a few tokens a request DRAM: 6.0 TB/s while keys are read (32
// requests of 5 tokens over 2k to 8k keys: 129 us, 110 of them). Over codes (145 us
// for the same) the chain of one query tile's scores, softmax and output, 3400
// clocks a tile, and the loading warps' 3600 beside it. 7 to 9 us pass until a
// CTA's first product (16 where keys are cut into chunks) and 4 us with each
// piece's start and end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_common.h"
#include "fa_extend_plan.cuh"
#include "fa_ptx.cuh"
#include "fa_tmap.h"

namespace fa {

static __device__ uint32_t g_extend_err;

namespace ext {

constexpr int BM = 128;     // rows a query tile
constexpr int ROWS = 256;   // rows an item
constexpr int RING = 8;     // piece descriptors in flight: K and V run at most three units ahead of what is issued
constexpr float RESCALE_LOG2 = 8.f;
constexpr float LN2 = 0.69314718055994531f;

// How K and V tiles reach shared memory.
enum Load : int { BOXES = 0, GATHER = 1, CODES = 2 };

template <int LOAD>
struct Threads {
  static constexpr int N = LOAD == BOXES ? 384 : 512;
  // readers of a piece: boxes or four loaders, Q, products, eight softmax warps
  static constexpr int READERS = (LOAD == BOXES ? 1 : 4) + 2 + 8;
};

template <int D, int LOAD>
struct Smem {
  static constexpr int PANELS = D / 64;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int TILE = BM * D * 2;
  static constexpr int PANEL = BM * 128;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * TILE;
  static constexpr int V_OFF = K_OFF + STAGES * TILE;
  static constexpr int PIECE_OFF = V_OFF + STAGES * TILE;
  static constexpr int BAR_OFF = PIECE_OFF + RING * static_cast<int>(sizeof(Piece));
  // q_full, q_empty, k0_full, kv_full[], kv_empty[], s_full[2], p_lo[2], p_hi[2], pv_done[2], o_free[2], final,
  // piece_full[], piece_empty[]
  static constexpr int NBARS = 3 + 2 * STAGES + 10 + 1 + 2 * RING;
  static constexpr int SLOT_OFF = BAR_OFF + NBARS * 8;
  static constexpr int PLAN_OFF = K_OFF;  // the plan is made before any K arrives
  static constexpr int RAW_OFF = (SLOT_OFF + 16 + 15) / 16 * 16;
  // 4-bit caches: a tile's codes and pairs of K and of V
  // Results pass through shared memory on their way out, OUT columns of a
  // warp's 32 rows at a time (as much as fits): rows of 16-byte pieces a thread
  // each, 32 rows to an instruction, took 2 us a piece.
  static constexpr int OUT_OFF = RAW_OFF + (LOAD == CODES ? 2 * TK * (D / 2 + D / 8) : 0);
  static constexpr int OUT = LOAD == CODES && D == 128 ? 16 : 64;
  static constexpr int BYTES = OUT_OFF + 8 * 32 * OUT * 2;
  // One CTA an SM (one 512-column TMEM allocation), 1024 bytes to align.
  static constexpr int ALLOC = BYTES + 1024 > 118784 ? BYTES + 1024 : 118784;
  static_assert(ALLOC <= 232448, "");
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barriers by their shared-memory address: in the softmax warps one base
// register serves them all.
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, uint32_t* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer();
    while (!(ok = mbar_try_wait(bar, parity)) && globaltimer() - t0 <= kWaitLimitNs) {
    }
    if (!ok) atomicExch(err, DEV_TIMEOUT);
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The ring of piece descriptors, as one reader sees it: a warp that reads
// every piece in order.
struct Pieces {
  Piece* ring;
  uint64_t *full, *empty;
  uint32_t* err;
  int next = 0;
  __device__ __forceinline__ Pieces(Piece* r, uint64_t* f, uint64_t* e, uint32_t* er)
      : ring(r), full(f), empty(e), err(er) {}
  __device__ __forceinline__ bool read(Piece* out) {
    const int s = next % RING;
    if (!mbar_wait_warp(&full[s], (next / RING) & 1, err)) return false;
    *out = ring[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
    ++next;
    return true;
  }
};

// Eight codes of one 32-bit word as bf16 values z + s (n − 8), one rounding
// each: a code lands in the mantissa of bf16 128, one subtraction leaves n − 8,
// exactly, and the fused multiply-add in bf16 rounds the sum.
__device__ __forceinline__ uint4 values8(uint32_t w, __nv_bfloat162 s, __nv_bfloat162 z) {
  const uint32_t v = w >> 4;
  const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(0xc308));  // -136
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t = __byte_perm(w, v, i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12));
    t = (t & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 n = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&t), off);
    const __nv_bfloat162 x = __hfma2(n, s, z);
    out[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A load that stays where it is written, a step before its value is used, and
// never under a branch: what a branch loads is copied where its paths meet, and
// the copy waits for the load.
__device__ __forceinline__ int load_entry(const int* p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// o = 0, lse = -inf for the rows of no request, dealt out to the whole grid:
// those before the first request and from the end of the last one on; where
// some request is taken for empty also the gaps between the others. gaps: NT
// places in shared memory.
template <int D, int NT>
__device__ __forceinline__ void zero_rows(const Extend& p, Requests<NT>* requests, PlanSmem* sm, int2* gaps, uint32_t* err) {
  const int tid = static_cast<int>(threadIdx.x);
  const bool ordered = !requests->disordered;
  const long long per = static_cast<long long>(p.H) * (D / 8), step = static_cast<long long>(gridDim.x) * NT;
  int covered = ordered ? p.q_starts[p.B] : 0;  // the end of the last request so far
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    if (!ordered) {
      const Request r = requests->tile(p, b0, sm);
      int all;
      const int before = block_max<NT>(r.n > 0 ? r.row0 + r.n : 0, sm->most, &all);
      gaps[tid] = r.n > 0 ? make_int2(max(covered, before), r.row0) : make_int2(0, 0);
      covered = max(covered, all);
      __syncthreads();
    }
    const bool last = ordered || b0 + NT >= p.B;
    const int n = ordered ? 1 : min(NT, p.B - b0);
    for (int i = 0; i < n + last; ++i) {
      const int2 gap = i == n ? make_int2(covered, p.T) : ordered ? make_int2(0, p.q_starts[0]) : gaps[i];
      const long long end = gap.y * per;
      for (long long at = gap.x * per + static_cast<long long>(blockIdx.x) * NT + tid; at < end; at += step) {
        if (in_range(at, 1, static_cast<long long>(p.T) * per, err))
          reinterpret_cast<uint4*>(p.o)[at] = make_uint4(0u, 0u, 0u, 0u);
        if (at % (D / 8) == 0 && in_range(at / (D / 8), 1, static_cast<long long>(p.T) * p.H, err))
          p.lse[at / (D / 8)] = -INFINITY;
      }
    }
    if (last) break;
    __syncthreads();  // the gaps are read
  }
}

template <int D, int LOAD, bool CHUNKS>
__global__ void __launch_bounds__(Threads<LOAD>::N, 1)
    extend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ Extend p) {
  using L = Smem<D, LOAD>;
  constexpr int ST = L::STAGES, NT = Threads<LOAD>::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + L::Q_OFF;
  uint8_t* sK = smem + L::K_OFF;
  uint8_t* sV = smem + L::V_OFF;
  Piece* ring = reinterpret_cast<Piece*>(smem + L::PIECE_OFF);
  // As in the forward, slot u % ST holds V of unit u and K of unit u + 1,
  // loaded and released together; the first unit's K has its own barrier.
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k0_full = q_full + 2;
  uint64_t* kv_full = q_full + 3;
  uint64_t* kv_empty = kv_full + ST;
  uint64_t* s_full = kv_empty + ST;    // [2], one per query tile
  uint64_t* p_lo = s_full + 2;         // [2] keys 0..63 of P
  uint64_t* p_hi = p_lo + 2;           // [2] keys 64..127
  uint64_t* pv_done = p_hi + 2;        // [2]
  uint64_t* o_free = pv_done + 2;      // [2] the epilogue has read O
  uint64_t* final_bar = o_free + 2;
  uint64_t* piece_full = final_bar + 1;
  uint64_t* piece_empty = piece_full + RING;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
  PlanSmem* plan_smem = reinterpret_cast<PlanSmem*>(smem + L::PLAN_OFF);
  uint32_t* err = &g_extend_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);
  launch_dependents();  // the merge may be set up; it waits for this grid's writes

  Requests<NT> requests(p, err);
  if (p.zero_skipped) zero_rows<D, NT>(p, &requests, plan_smem, reinterpret_cast<int2*>(plan_smem + 1), err);

  Shape<CHUNKS> sh{2 * p.tpt, p.causal, p.lc, 0};
  Cut cut;
  Place at;
  i64 items0;
  if (!plan<NT, false>(p, &requests, &sh, plan_smem, cta, &cut, &at, &items0)) {
    if (threadIdx.x == 0 && in_range(cta, 1, p.ctas, err)) p.cuts[cta].parts = 0;
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(k0_full, LOAD == BOXES ? 1 : LOAD == GATHER ? 128 : 4);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kv_full[s], LOAD == BOXES ? 1 : LOAD == GATHER ? 128 : 4);
      mbar_init(&kv_empty[s], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_lo[g], 4);
      mbar_init(&p_hi[g], 4);
      mbar_init(&pv_done[g], 1);
      mbar_init(&o_free[g], 4);
    }
    mbar_init(final_bar, 1);
    for (int i = 0; i < RING; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], Threads<LOAD>::READERS);
    }
    fence_mbar_init();
  }
  // Rows of a query tile that no token fills (128 is no multiple of the heads)
  // are zero for good: their scores then never ask for a rescaling.
  const int filled = p.tpt * p.heads;
  if (filled < BM)
    for (int i = threadIdx.x; i < 2 * L::PANELS * (BM - filled) * 8; i += NT) {
      const int panel = i / ((BM - filled) * 8), rest = i % ((BM - filled) * 8);
      *reinterpret_cast<uint4*>(sQ + panel * L::PANEL + filled * 128 + rest * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  fence_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The launch's registers go where they are needed: 128 · (104 + 2 · 200) of
  // 384 · 168 with boxes, else 128 · (88 + 2 · 176 + 72) = 512 · 128. (Softmax at
  // 160: 679 us for 300 tokens at 131072 keys over codes, not 587.)
  if (warp < 4) {
    regs_down<LOAD == BOXES ? 104 : 88>();
    if (warp == 0) {
      // --------------------------------------------------------------- pieces
      locate(p, sh, cut.start(cta), &at);
      int idx = 0;
      auto emit = [&](Piece x) {
        const int s = idx % RING;
        if (x.slot >= p.n_slots) {  // the host's bound holds: never
          atomicExch(err, DEV_BOUNDS);
          x.slot = 2 * cta;
        }
        if (idx >= RING && !mbar_wait_warp(&piece_empty[s], ((idx / RING) - 1) & 1, err)) return false;
        if (lane == 0) {
          ring[s] = x;
          mbar_arrive(&piece_full[s]);
        }
        __syncwarp();
        ++idx;
        return true;
      };
      ItemCut entered{};
      if (walk(p, sh, cut, cta, at, &entered, emit)) emit(Piece{});
      if (lane == 0 && in_range(cta, 1, p.ctas, err)) p.cuts[cta] = entered;
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16(BM, TK, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(BM, D, false, true);
      const uint64_t dq = sdesc_kmajor(smem_u32(sQ), 0);
      const uint64_t dk = sdesc_kmajor(smem_u32(sK), 0);
      const uint64_t dv = sdesc_mnmajor(smem_u32(sV), 0, L::PANEL);
      auto issue_s = [&](int g, int s) {  // S_g = Q_g Kᵀ, K in stage s
        const uint64_t a = desc_add(dq, g * L::TILE), b = desc_add(dk, s * L::TILE);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss(tmem + g * TK, desc_add(a, kmajor_step(ks, L::PANEL)), desc_add(b, kmajor_step(ks, L::PANEL)),
                   idesc_s, ks > 0);
          tc_commit(&s_full[g]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int g, int s, int half, uint32_t acc0) {  // O_g += P_g V over 64 keys
        const uint64_t b = desc_add(dv, s * L::TILE);
        if (elect_one()) {
#pragma unroll
          for (int k4 = 0; k4 < TK / 32; ++k4) {
            const int ks = half * (TK / 32) + k4;
            mma_ts(tmem + 256 + g * 128, tmem + g * TK + ks * 8, desc_add(b, mnmajor_step(ks)), idesc_o,
                   ks > 0 ? 1u : acc0);
          }
          if (half == 1) tc_commit(&pv_done[g]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) tc_commit(bar);
        __syncwarp();
      };
      Pieces pieces(ring, piece_full, piece_empty, err);
      Piece x;
      // (A share may lie within one tile: then there is no piece.)
      bool ok = pieces.read(&x) && x.n > 0 && mbar_wait_warp(q_full, 0, err) && mbar_wait_warp(k0_full, 0, err);
      int n[2] = {0, 0}, seen[2] = {0, 0}, done[2] = {0, 0};  // tiles of the piece; units, pieces so far of each query tile
      int len = 0, idx = 0, u = 0;
      auto first_s = [&](int s) {  // the scores of a piece's first unit
        n[0] = x.n0, n[1] = x.n1;
        if (n[0] > 0) issue_s(0, s);
        if (n[1] > 0) issue_s(1, s);
      };
      if (ok) {
        tc_fence_after();
        if (LOAD == GATHER) fence_async_smem();
        len = x.n;
        first_s(0);
        commit(&kv_empty[ST - 1]);  // the first K is read: slot ST - 1 may load
        if (len == 1) commit(q_empty);
      }
      while (ok && len > 0) {
        int next = 0;
        for (int j = 0; j < len && ok; ++j, ++u) {
          const int s = u % ST, s1 = (u + 1) % ST;
          const bool last = j + 1 == len;
          ok = mbar_wait_warp(&kv_full[s], (u / ST) & 1, err);
          if (!ok) break;
          if (LOAD == GATHER) fence_async_smem();  // the lanes' copies, for the tensor core
          auto pv = [&](int g, bool begun) {  // O_g (+)= P_g V, half by half as P arrives
            if (!begun && done[g] > 0 && !mbar_wait_warp(&o_free[g], (done[g] - 1) & 1, err)) return false;
            if (!mbar_wait_warp(&p_lo[g], seen[g] & 1, err)) return false;
            tc_fence_after();
            issue_pv(g, s, 0, begun ? 1u : 0u);
            if (!mbar_wait_warp(&p_hi[g], seen[g] & 1, err)) return false;
            tc_fence_after();
            issue_pv(g, s, 1, 1u);
            ++seen[g];
            return true;
          };
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (j >= n[g]) continue;
            ok = pv(g, j > 0);
            if (!ok) break;
            if (j + 1 < n[g]) issue_s(g, s1);
          }
          if (!ok) break;
          if (j + 2 == len) commit(q_empty);  // the piece's last scores are under way
          if (last) {
            if (n[0] > 0) ++done[0];
            if (n[1] > 0) ++done[1];
            ok = pieces.read(&x);
            if (!ok) break;
            next = x.n;
            if (next > 0) {
              ok = mbar_wait_warp(q_full, (idx + 1) & 1, err);
              if (!ok) break;
              tc_fence_after();
              first_s(s1);
              if (next == 1) commit(q_empty);
            }
          }
          commit(&kv_empty[s]);  // V of unit u and K of unit u + 1 are read
        }
        len = next;
        ++idx;
      }
      commit(final_bar);
      mbar_wait_warp(final_bar, 0, err);
    } else if (warp == 3) {
      // -------------------------------------------------------------- Q tiles
      if (lane == 0) prefetch_tmap(&tq);
      const int bytes = p.tpt * p.heads * 128 * L::PANELS;
      Pieces pieces(ring, piece_full, piece_empty, err);
      Piece x;
      int idx = 0;
      for (; pieces.read(&x) && x.n > 0; ++idx) {
        if (idx > 0 && !mbar_wait_warp(q_empty, (idx - 1) & 1, err)) break;
        if (lane == 0) {
          const int tiles = (x.n0 > 0) + (x.n1 > 0);
          if (tiles == 0) mbar_arrive(q_full);
          else mbar_arrive_expect_tx(q_full, tiles * bytes);
          for (int g = 0; g < 2; ++g)
            if ((g ? x.n1 : x.n0) > 0)
              for (int c = 0; c < L::PANELS; ++c)
                tma_load_3d(sQ + g * L::TILE + c * L::PANEL, &tq, q_full, c * 64, x.head0, x.tok0 + g * p.tpt);
        }
        __syncwarp();
      }
      if (idx > 0) mbar_wait_warp(q_full, (idx - 1) & 1, err);  // no copy outlives the CTA
    } else if (LOAD == BOXES) {
      // --------------------------------------------------- K and V by TMA boxes
      // Lane i issues the box of block i of a tile; a block past the context or
      // outside the cache is asked for at an out-of-range coordinate, which
      // reads zeros. Table entries are loaded two units ahead.
      if (lane == 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
      }
      const int bpt = TK / p.bs;
      struct Unit {
        bool any, want;  // a unit; this lane has a box of the context
        int entry, kvh;  // this lane's table entry
      };
      Pieces pieces(ring, piece_full, piece_empty, err);
      Piece x;
      x.n = 0;
      int j = 0;
      bool more = true;
      auto fetch = [&]() -> Unit {  // the next unit
        if (more && ++j >= x.n) {
          more = pieces.read(&x) && x.n > 0;
          j = 0;
        }
        const int bi = (x.kt0 + j) * bpt + lane;
        Unit t;
        t.any = more;
        t.want = more && lane < bpt && static_cast<long long>(bi) * p.bs < x.len;
        t.kvh = x.kvh;
        const long long ti = t.want ? static_cast<long long>(x.b) * p.max_blocks + bi : 0;
        t.want = t.want && in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err);
        t.entry = load_entry(p.block_table + (t.want ? ti : 0));
        return t;
      };
      auto place = [&](const Unit& t) {  // the box's outer coordinate
        if (t.want && t.entry >= 0 && t.entry < p.num_blocks) return t.entry * p.Hkv + t.kvh;
        if (t.want) atomicExch(err, DEV_BAD_INDEX);
        return p.num_blocks * p.Hkv;
      };
      auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int z) {
        if (lane < bpt)
          for (int c = 0; c < L::PANELS; ++c) tma_load_3d(dst + c * L::PANEL + lane * p.bs * 128, map, bar, c * 64, 0, z);
      };
      Unit cur = fetch();
      int z = place(cur), u = 0;
      bool ok = cur.any;
      if (ok) {
        if (lane == 0) mbar_arrive_expect_tx(k0_full, L::TILE);
        __syncwarp();
        load(&tk, sK, k0_full, z);
      }
      Unit nxt = fetch(), far = fetch();
      while (ok) {
        const int s = u % ST, s1 = (u + 1) % ST;
        const int z1 = nxt.any ? place(nxt) : 0;
        if (u >= ST - 1) ok = mbar_wait_warp(&kv_empty[s], ((u - (ST - 1)) / ST) & 1, err);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], nxt.any ? 2 * L::TILE : L::TILE);
        __syncwarp();
        load(&tv, sV + s * L::TILE, &kv_full[s], z);
        ++u;
        if (!nxt.any) break;
        load(&tk, sK + s1 * L::TILE, &kv_full[s], z1);
        z = z1;
        nxt = far;
        far = fetch();
      }
      // no copy outlives the CTA
      if (cur.any) mbar_wait_warp(k0_full, 0, err);
      for (int i = max(0, u - ST); i < u; ++i) mbar_wait_warp(&kv_full[i % ST], (i / ST) & 1, err);
    }
  } else if (warp < 12) {
    regs_up<LOAD == BOXES ? 200 : 176>();
    // -------------------------------------------------------------- softmax
    const int g = (warp - 4) >> 2;  // query tile
    const int quarter = warp & 3;   // TMEM lanes 32*quarter .. +31
    const int r = quarter * 32 + lane;
    const uint32_t s_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + g * TK;
    const uint32_t bars = smem_u32(s_full + g);  // s_full[g]; p_lo, p_hi, pv_done and o_free follow, two by two
    constexpr uint32_t P_LO = 16, P_HI = 32, PV_DONE = 48, O_FREE = 64;
    const uint32_t o_addr = s_addr + 256;
    const float scale_log2 = p.scale_log2;
    // Registers are short here (a row's 128 scores are in them): what a row
    // needs of its piece is read from the ring each time, where the piece stays
    // until this warp is through with it.
    struct Row {  // this thread's row
      bool valid;
      int tok, head;  // token of the item, head of the K/V head's
    };
    auto row_of = [&](const Piece& x) {
      const int tt = r / p.heads;
      Row y{false, g * p.tpt + tt, r - tt * p.heads};
      y.valid = r < filled && y.tok < x.ntok && y.head < x.heads;
      return y;
    };
    constexpr int ALL = 0x7fffffff;
    auto sight_of = [&](const Piece& x) {  // keys this row sees (a row without a token: ALL)
      const Row y = row_of(x);
      return !y.valid ? ALL : p.causal ? max(x.pos0 + y.tok + 1, 0) : x.len;
    };
    int seen = 0;  // units of this group
    for (int idx = 0;; ++idx) {
      if (!mbar_wait_warp(&piece_full[idx % RING], (idx / RING) & 1, err)) break;
      const Piece& x = ring[idx % RING];
      if (x.n == 0) break;
      bool ok = true;
      const int sight_lo = __reduce_min_sync(0xffffffffu, sight_of(x));  // ALL: no row of the warp has a token
      float m = -INFINITY;  // exponent reference (log2 units of scaled scores)
      float l = 0.f;        // running denominator relative to m
      const bool live = sight_lo != ALL;
      const int edge = min(sight_lo, x.len);  // keys below it need no mask and no zeroed values
      const int k_end = (x.kt0 + (g ? x.n1 : x.n0)) * TK;
      bool begun = false;
      for (int k0 = x.kt0 * TK; k0 < k_end; k0 += TK, ++seen) {
        ok = wait_at(bars, seen & 1, err);
        if (!ok) break;
        tc_fence_after();
        // A box brings whole cache blocks: slots past the context may hold
        // anything, and a NaN of theirs would outlive its zero probability.
        // Their value rows are zeroed before the product reads them. (S of this
        // unit is there, so the barrier is at this unit's phase at least: its
        // parity wait is exact.)
        if (LOAD == BOXES && k0 + TK > edge && k0 + TK > x.len) {
          const int u = x.unit0 + k0 / TK - x.kt0, s = u % ST;
          ok = mbar_wait_warp(&kv_full[s], (u / ST) & 1, err);
          if (!ok) break;
          if (k0 + r >= x.len)
            for (int i = 0; i < L::PANELS * 8; ++i)
              *reinterpret_cast<uint4*>(sV + s * L::TILE + (i >> 3) * L::PANEL + r * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
        }
        auto release = [&](uint32_t bar) {  // this half of P is in TMEM
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(bars + bar);
        };
        if (!live) {  // no row to compute: what P holds for these rows reaches no other
          release(P_LO);
          release(P_HI);
          continue;
        }
        uint32_t raw[4][32];
        tmem_ld32(s_addr + 0, raw[0]);
        tmem_ld32(s_addr + 32, raw[1]);
        tmem_ld32(s_addr + 64, raw[2]);
        tmem_ld32(s_addr + 96, raw[3]);
        tmem_ld_wait();
        float y[TK];
#pragma unroll
        for (int c = 0; c < TK; ++c) y[c] = __uint_as_float(raw[c / 32][c % 32]);
        if (k0 + TK > edge) {
          const int mine = sight_of(x) - k0;
#pragma unroll
          for (int c = 0; c < TK; ++c)
            if (c >= mine) y[c] = -INFINITY;
        }
        float2 sum[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] = make_float2(0.f, 0.f);
        const float2 sc2 = make_float2(scale_log2, scale_log2);
        // P is rounded to bf16, half a step (2^-8 of a weight) at most, as in the
        // forward; its sum is that of the unrounded weights. Results are 1.2 to 1.4
        // times as far from 64 bits as their own rounding. The remainder as a second
        // bf16 number and product would cost a third more time and up to two thirds
        // over codes: a prompt of 8192 tokens 539 us and not 404, 2777 tokens of 12
        // requests 269 and not 212, over codes 373 and not 255.
        auto p_chunk = [&](int c, float2 nm2) {
          uint32_t pk[16];
#pragma unroll
          for (int t2 = 0; t2 < 16; ++t2) {
            const float2 e = ffma2(make_float2(y[c + 2 * t2], y[c + 2 * t2 + 1]), sc2, nm2);
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            sum[t2 & 3] = fadd2(sum[t2 & 3], make_float2(p0, p1));
            pk[t2] = pack_bf16x2(p0, p1);
          }
          tmem_st16(s_addr + c / 2, pk);
        };
        // The first half against the reference so far, before the tile's
        // maximum is known; again if that outgrew it (as in the forward).
        auto minus = [&]() {  // -m; 0 for a row that has seen no key: 2^-inf = 0 throughout
          const float v = m == -INFINITY ? 0.f : -m;
          return make_float2(v, v);
        };
        // (One copy of the two chunks' code, for the first time and again: beside
        // the other warps' it has to stay in the instruction cache.)
        bool again = false;
#pragma unroll 1
        while (true) {
          if (begun || again) {
            p_chunk(0, minus());
            p_chunk(32, minus());
          }
          if (again) break;
          float mx[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx[q] = fmaxf(y[q], y[8 + q]);
#pragma unroll
          for (int c = 16; c < TK; c += 16)
#pragma unroll
            for (int q = 0; q < 8; ++q) mx[q] = fmax3(mx[q], y[c + q], y[c + 8 + q]);
          const float tile_max = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * scale_log2;
          const bool raise = __any_sync(0xffffffffu, tile_max > m + RESCALE_LOG2);
          if (!raise && begun) break;
          const float m_new = fmaxf(m, tile_max);
          const float alpha = m_new == -INFINITY ? 1.f : ex2(m - m_new);  // 0 on a row's first key
          m = m_new;
          l *= alpha;
          if (begun) {
            ok = wait_at(bars + PV_DONE, (seen - 1) & 1, err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_addr + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int t2 = 0; t2 < 16; ++t2) o[t2] = __float_as_uint(__uint_as_float(o[t2]) * alpha);
              tmem_st16(o_addr + c, o);
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[q] = make_float2(0.f, 0.f);
          again = true;
        }
        if (!ok) break;
        release(P_LO);
        p_chunk(64, minus());
        p_chunk(96, minus());
        release(P_HI);
        begun = true;
        l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
      }
      if (!ok) break;
      // ------------------------------------------------------------ epilogue
      const bool any = (g ? x.n1 : x.n0) > 0;
      if (any) {
        ok = wait_at(bars + PV_DONE, (seen - 1) & 1, err);
        if (!ok) break;
        tc_fence_after();
      }
      const bool none = l == 0.f;               // no key: nothing of O, whatever it holds
      const float inv = none ? 0.f : 1.f / l;   // NaN stays NaN
      const float lse = none ? -INFINITY : (m + __log2f(l)) * LN2;
      const Row y = row_of(x);
      const bool valid = y.valid;
      const int orow = (x.tok0 + y.tok) * p.H + x.head0 + y.head;  // below T·H, if valid
      const long long prow = static_cast<long long>(x.slot) * ROWS + g * BM + r;
      constexpr int CW = 16;  // columns at a time
      float f[CW];
      auto columns = [&](int c) {  // this row's results c .. c + CW - 1
#pragma unroll
        for (int i = 0; i < CW; ++i) f[i] = 0.f;
        if (!any) return;
        uint32_t o[CW];
        tmem_ld16(o_addr + c, o);
        tmem_ld_wait();
        if (!none) {
#pragma unroll
          for (int i = 0; i < CW; ++i) f[i] = __uint_as_float(o[i]) * inv;
        }
        __syncwarp();
      };
      if (!live) {  // no row of a token
      } else if (x.slot < 0) {
        uint8_t* out = smem + L::OUT_OFF + (warp - 4) * (32 * L::OUT * 2);
        constexpr int CH = L::OUT / 8, RPI = 32 / CH;  // 16-byte pieces of a row; rows to an instruction
        const int at_row = valid ? orow : -1;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += L::OUT) {
#pragma unroll 1
          for (int c = 0; c < L::OUT; c += CW) {
            columns(c0 + c);
#pragma unroll
            for (int e = 0; e < CW / 8; ++e) {
              const float* v = f + e * 8;
              *reinterpret_cast<uint4*>(out + lane * (L::OUT * 2) + (((c / 8 + e) ^ (lane & (CH - 1))) << 4)) =
                  make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            const int rr = k * RPI + lane / CH, ch = lane % CH;
            const int to = __shfl_sync(0xffffffffu, at_row, rr);
            const uint4 v = *reinterpret_cast<const uint4*>(out + rr * (L::OUT * 2) + ((ch ^ (rr & (CH - 1))) << 4));
            const long long off = static_cast<long long>(to) * D + c0 + ch * 8;
            if (to >= 0 && in_range(off, 8, static_cast<long long>(p.T) * p.H * D, err))
              *reinterpret_cast<uint4*>(p.o + off) = v;
          }
          __syncwarp();
        }
        if (valid && in_range(orow, 1, static_cast<long long>(p.T) * p.H, err)) p.lse[orow] = lse;
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += CW) {
          columns(c);
          if (valid) {
#pragma unroll
            for (int e = 0; e < CW / 4; ++e) {
              const long long off = ((static_cast<long long>(x.slot) * (D / 4) + c / 4 + e) * ROWS + g * BM + r) * 4;
              if (in_range(off, 4, static_cast<long long>(p.n_slots) * ROWS * D, err))
                *reinterpret_cast<float4*>(p.o_part + off) = make_float4(f[e * 4], f[e * 4 + 1], f[e * 4 + 2], f[e * 4 + 3]);
            }
          }
          __syncwarp();
        }
        if (valid && in_range(prow, 1, static_cast<long long>(p.n_slots) * ROWS, err)) p.lse_part[prow] = lse;
      }
      if (any) {  // O is read: the next piece's products may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(bars + O_FREE);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[idx % RING]);
    }
  } else if constexpr (LOAD != BOXES) {
    regs_down<72>();
    // ----------------------------------------- K and V row by row, or unpacked
    // Each of four warps takes 32 rows of a tile, lane i the place of row i.
    constexpr uint32_t NO_ROW = 0xffffffffu;  // zeros (the host keeps the cache below 2^32 - 1 rows)
    const int w = warp - 12;
    const long long rows_all = static_cast<long long>(p.num_blocks) * p.Hkv * p.bs;
    struct Unit {
      bool any;
      uint32_t row;
    };
    struct Raw {  // a unit's row before its table entry is there
      bool any, want;
      int entry, kvh, slot;
    };
    Pieces pieces(ring, piece_full, piece_empty, err);
    Piece x;
    x.n = 0;
    int j = 0;
    bool more = true;
    auto fetch = [&]() -> Raw {
      if (more && ++j >= x.n) {
        more = pieces.read(&x) && x.n > 0;
        j = 0;
      }
      const int key = (x.kt0 + j) * TK + w * 32 + lane;
      Raw t;
      t.any = more;
      t.want = more && key < x.len;
      const int bi = p.block_of(t.want ? key : 0);
      t.kvh = x.kvh;
      t.slot = key - bi * p.bs;
      const long long ti = static_cast<long long>(t.want ? x.b : 0) * p.max_blocks + bi;
      t.want = t.want && in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err);
      t.entry = load_entry(p.block_table + (t.want ? ti : 0));
      return t;
    };
    auto resolve = [&](const Raw& t) -> Unit {
      Unit y{t.any, NO_ROW};
      if (t.want) {
        if (t.entry >= 0 && t.entry < p.num_blocks)
          y.row = (static_cast<uint32_t>(t.entry) * static_cast<uint32_t>(p.Hkv) + static_cast<uint32_t>(t.kvh)) *
                      static_cast<uint32_t>(p.bs) + static_cast<uint32_t>(t.slot);
        else
          atomicExch(err, DEV_BAD_INDEX);
      }
      return y;
    };
    int u = 0;
    if constexpr (LOAD == GATHER) {
      auto copy = [&](const void* cache, uint8_t* dst, uint32_t row) {
        constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks a row, rows a step
        const int c = lane % CH, sub = lane / CH;
#pragma unroll 4
        for (int k = 0; k < CH; ++k) {
          const int r = k * RPI + sub;
          const uint32_t at_row = __shfl_sync(0xffffffffu, row, r);
          const bool live = at_row != NO_ROW && in_range(at_row, 1, rows_all, err);
          const char* src = static_cast<const char*>(cache) + static_cast<size_t>(live ? at_row : 0u) * (D * 2) + c * 16;
          cp_async_16(dst + (c >> 3) * L::PANEL + (w * 32 + r) * 128 + (((c & 7) ^ (r & 7)) << 4), src, live ? 16u : 0u);
        }
      };
      Raw a = fetch(), b = fetch();
      Unit cur = resolve(a);
      bool ok = cur.any;
      if (ok) {
        copy(p.k_cache, sK, cur.row);
        cp_async_arrive_noinc(k0_full);
      }
      a = b, b = fetch();
      while (ok) {
        const int s = u % ST, s1 = (u + 1) % ST;
        const Unit nxt = resolve(a);
        if (u >= ST - 1) ok = mbar_wait_warp(&kv_empty[s], ((u - (ST - 1)) / ST) & 1, err);
        if (!ok) break;
        copy(p.v_cache, sV + s * L::TILE, cur.row);
        if (nxt.any) copy(p.k_cache, sK + s1 * L::TILE, nxt.row);
        cp_async_arrive_noinc(&kv_full[s]);
        ++u;
        if (!nxt.any) break;
        cur = nxt;
        a = b, b = fetch();
      }
      cp_async_commit();
      cp_async_wait<0>();  // no copy outlives the CTA
    } else {
      // A lane takes 32 codes (16 bytes) of a row and their group's pair. They
      // wait in shared memory, in a place of the lane's own, for the step they
      // are unpacked in: the copies of the next tile are under way meanwhile.
      // (Held in registers instead, a tile took 6000 clocks: the compiler's waits
      // for one load cover others. Now 3600 to 4200, 1100 to 1400 of them for
      // each of keys and values: 4.25 instructions a pair of values, at half rate.)
      constexpr int CPR = D / 32, RPI = 32 / CPR;  // 16-byte pieces a row, rows a step; CPR steps
      const int quarter = lane % CPR, sub = lane / CPR;
      uint8_t* kraw = smem + L::RAW_OFF + w * (2 * CPR * 32 * 20) + lane * 16;
      uint8_t* vraw = kraw + CPR * 32 * 20;
      constexpr int PAIRS = CPR * 32 * 16;  // the pairs stand behind the codes, 4 bytes a lane
      auto fetch_codes = [&](const void* cache, const uint32_t* scale, const Unit& t, uint8_t* raw) {
#pragma unroll
        for (int k = 0; k < CPR; ++k) {
          const uint32_t row = __shfl_sync(0xffffffffu, t.row, k * RPI + sub);
          const bool live = row != NO_ROW && in_range(row, 1, rows_all, err);  // else zeros: step and centre 0
          const size_t at_row = live ? row : 0u;
          cp_async_16(raw + k * 512, static_cast<const uint8_t*>(cache) + at_row * (D / 2) + quarter * 16, live ? 16u : 0u);
          cp_async_4(raw + PAIRS + k * 128 - lane * 12, scale + at_row * (D / 64) + quarter / 2, live ? 4u : 0u);
        }
        cp_async_commit();
      };
      // Rows r and r + 1 and both panels meet in one store: with the words of
      // the second panel's lanes two places on, no two lanes share a bank.
      const bool swap = quarter & 2;
      uint32_t put[4];  // where a step's words go: row `sub` of it (rows a step on are RPI · 128 bytes on)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        put[e] = (quarter >> 1) * L::PANEL + (w * 32 + sub) * 128 +
                 ((((quarter & 1) * 4 + (e ^ (swap ? 2 : 0))) ^ (sub & 7)) << 4);
      auto unpack = [&](uint8_t* dst, const uint8_t* raw) {
        uint4 c = *reinterpret_cast<const uint4*>(raw);
        uint32_t pair = *reinterpret_cast<const uint32_t*>(raw + PAIRS - lane * 12);
        // Two steps at a time: four do not stay in the instruction cache beside the
        // softmax (2777 tokens of 12 requests: one 249 us, two 244, four 250; 32
        // requests of 5 tokens 148, 146 and 158).
#pragma unroll 2
        for (int k = 0; k < CPR; ++k) {
          const uint32_t sbits = __byte_perm(pair, 0, 0x1010), zbits = __byte_perm(pair, 0, 0x3232);
          const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&sbits);
          const __nv_bfloat162 z2 = *reinterpret_cast<const __nv_bfloat162*>(&zbits);
          const uint32_t word[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
          if (k + 1 < CPR) {
            c = *reinterpret_cast<const uint4*>(raw + (k + 1) * 512);
            pair = *reinterpret_cast<const uint32_t*>(raw + PAIRS + (k + 1) * 128 - lane * 12);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(dst + put[e] + k * (RPI * 128)) = values8(word[e], s2, z2);
        }
      };
      auto publish = [&](uint64_t* bar) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      // K of unit u + 1 and V of unit u, copied a step ahead.
      Raw a = fetch(), b = fetch();
      Unit cur = resolve(a);
      fetch_codes(p.k_cache, p.k_scale, cur, kraw);
      fetch_codes(p.v_cache, p.v_scale, cur, vraw);
      Unit nxt = resolve(b);
      Raw far = fetch();
      bool ok = cur.any;
      cp_async_wait<1>();
      if (ok) {
        unpack(sK, kraw);
        publish(k0_full);
      }
      fetch_codes(p.k_cache, p.k_scale, nxt, kraw);
      while (ok) {
        const int s = u % ST, s1 = (u + 1) % ST;
        const Unit after = resolve(far);
        far = fetch();
        if (u >= ST - 1) ok = mbar_wait_warp(&kv_empty[s], ((u - (ST - 1)) / ST) & 1, err);
        if (!ok) break;
        cp_async_wait<1>();
        unpack(sV + s * L::TILE, vraw);
        fetch_codes(p.v_cache, p.v_scale, nxt, vraw);
        cp_async_wait<1>();
        if (nxt.any) unpack(sK + s1 * L::TILE, kraw);
        fetch_codes(p.k_cache, p.k_scale, after, kraw);
        publish(&kv_full[s]);
        ++u;
        if (!nxt.any) break;
        nxt = after;
      }
      cp_async_wait<0>();  // no copy outlives the CTA
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- merge
//
// One output row from its parts: lse = ln Σ_s e^(lse_s), o = Σ_s e^(lse_s −
// lse) o_s. The first ctas - 1 blocks take the items that shares cut: a CTA
// whose share begins within an item has noted it (worked out from the lengths
// again they took 6 us more), and the blocks of an item's CTAs but the first
// deal its rows out among them. (All by one block: 152 us for 64 tokens at
// 131072 keys, 8 items of 19 parts each; now 121.) The others take one long item
// each.
constexpr int MERGE_THREADS = 512;

// An item's rows: 32 rows and W 4-value groups of columns a task, UNROLL parts at a time.
template <int D, int W, int UNROLL>
__device__ __forceinline__ void merge_rows(const Extend& p, const ItemCut& it, const int* parts, int first, int step,
                                           uint32_t* err) {
  const int lane = threadIdx.x & 31, n = it.parts;
  constexpr int ACROSS = D / 4 / W, TASKS = ROWS / 32 * ACROSS;
  for (int task = first; task < TASKS; task += step) {
    const int row = task / ACROSS * 32 + lane, c0 = task % ACROSS * W, g = row / BM, r = row % BM;
    const int tt = r / p.heads, hh = r - tt * p.heads, tok = g * p.tpt + tt;
    if (r >= p.tpt * p.heads || tok >= it.ntok || hh >= it.heads) continue;
    float m = -INFINITY;
#pragma unroll UNROLL
    for (int s = 0; s < n; ++s) {
      const long long pr = static_cast<long long>(parts[s]) * ROWS + row;
      const float v = in_range(pr, 1, static_cast<long long>(p.n_slots) * ROWS, err) ? p.lse_part[pr] : 0.f;
      m = v != v || m != m ? NAN : fmaxf(m, v);  // a part whose lse is NaN makes its row NaN
    }
    float l = 0.f;
    float4 acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m != -INFINITY) {
#pragma unroll UNROLL
      for (int s = 0; s < n; ++s) {
        const long long pr = static_cast<long long>(parts[s]) * ROWS + row;
        const float v = in_range(pr, 1, static_cast<long long>(p.n_slots) * ROWS, err) ? p.lse_part[pr] : 0.f;
        const float w = ex2((v - m) * 1.4426950408889634f);
        l += w;
        float4 t[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const long long off = ((static_cast<long long>(parts[s]) * (D / 4) + c0 + i) * ROWS + row) * 4;
          t[i] = in_range(off, 4, static_cast<long long>(p.n_slots) * ROWS * D, err)
                     ? *reinterpret_cast<const float4*>(p.o_part + off) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          acc[i].x = fmaf(w, t[i].x, acc[i].x), acc[i].y = fmaf(w, t[i].y, acc[i].y);
          acc[i].z = fmaf(w, t[i].z, acc[i].z), acc[i].w = fmaf(w, t[i].w, acc[i].w);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long orow = static_cast<long long>(it.tok0 + tok) * p.H + it.head0 + hh;
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const long long off = orow * D + (c0 + i) * 4;
      if (in_range(off, 8, static_cast<long long>(p.T) * p.H * D, err))
        *reinterpret_cast<uint4*>(p.o + off) =
            make_uint4(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv),
                       pack_bf16x2(acc[i + 1].x * inv, acc[i + 1].y * inv), pack_bf16x2(acc[i + 1].z * inv, acc[i + 1].w * inv));
    }
    if (c0 == 0 && in_range(orow, 1, static_cast<long long>(p.T) * p.H, err))
      p.lse[orow] = l == 0.f ? -INFINITY : m + __logf(l);
  }
}

// (", 1": left to itself the compiler takes 64 registers and spills.)
template <int D, bool CHUNKS>
__global__ void __launch_bounds__(MERGE_THREADS, 1) extend_merge_kernel(const __grid_constant__ Extend p) {
  __shared__ int parts[MAX_PARTS];
  __shared__ ItemCut shared_item;
  uint32_t* err = &g_extend_err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int job = static_cast<int>(blockIdx.x);
  if (!CHUNKS || job < p.ctas - 1) {
    wait_for_primary();
    if (threadIdx.x == 0) shared_item = in_range(job + 1, 1, p.ctas, err) ? p.cuts[job + 1] : ItemCut{};
    __syncthreads();
    const int first = job + 1 - shared_item.nth;
    for (int i = threadIdx.x; i < shared_item.parts; i += MERGE_THREADS) parts[i] = i == 0 ? 2 * first + 1 : 2 * (first + i);
  } else if constexpr (CHUNKS) {
    __shared__ PlanSmem plan_smem;
    Shape<true> sh{2 * p.tpt, p.causal, p.lc, 0};
    Cut cut;
    Place at;
    i64 items0;
    const int want = job - (p.ctas - 1);
    if (threadIdx.x == 0) shared_item = ItemCut{};
    Requests<MERGE_THREADS> requests(p, err);
    if (plan<MERGE_THREADS, true>(p, &requests, &sh, &plan_smem, want, &cut, &at, &items0) && warp == 0) {
      const int first = sh.first_long(at.r, 0), each = at.r.items - first;
      const int nth = static_cast<int>(want - items0);
      at.hv = nth / each;
      at.i = first + nth % each;
      const int n_c = (sh.keys(at.r, at.i) + sh.lc - 1) / sh.lc;
      int n = 0;
      for (int c0 = 0; c0 < n_c; c0 += 32) {
        at.c = c0 + lane;
        int mine = 0, k = 0;
        if (at.c < n_c) {
          const i64 row = sh.costs_before(at.r, at.c, at.r.items);
          at.item0 = at.request0 + sh.chunks_before(at.r, at.c) * p.hv + row * at.hv + sh.costs_before(at.r, at.c, at.i);
          k = cut.owner(at.item0);
          mine = parts_of(p, sh, cut, at, k, [](int, int) {});
        }
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += t;
        }
        const int at0 = n + sum - mine;
        if (mine > 0)
          parts_of(p, sh, cut, at, k, [&](int i, int slot) {
            if (slot >= p.n_slots) {  // the host's bound holds: never
              atomicExch(err, DEV_BOUNDS);
              slot = 0;
            }
            if (at0 + i < MAX_PARTS) parts[at0 + i] = slot;
          });
        n += __shfl_sync(0xffffffffu, sum, 31);
      }
      const int per = p.hv / p.Hkv, h0 = at.hv % per * p.heads, G = p.H / p.Hkv, t0 = at.i * sh.span;
      if (lane == 0)
        shared_item = ItemCut{min(n, MAX_PARTS), 0, at.r.row0 + t0, min(sh.span, at.r.n - t0), at.hv / per * G + h0,
                              min(p.heads, G - h0)};
    }
    wait_for_primary();
  }
  __syncthreads();
  const ItemCut it = shared_item;
  if (it.parts == 0) return;
  const int blocks = it.nth > 0 ? it.parts - 1 : 1, block = max(it.nth - 1, 0);
  const int first = block * (MERGE_THREADS / 32) + warp, step = blocks * (MERGE_THREADS / 32);
  // A warp takes 32 rows and a quarter of the columns at a time; 8 columns where
  // that leaves half the warps without a task (items in many parts or with few rows).
  const int rows0 = min(it.ntok, p.tpt) * p.heads, rows1 = max(it.ntok - p.tpt, 0) * p.heads;
  if (2 * blocks >= (rows0 + 31) / 32 + (rows1 + 31) / 32)
    merge_rows<D, 2, 2>(p, it, parts, first, step, err);
  else
    merge_rows<D, D / 16, 2>(p, it, parts, first, step, err);
}

// ------------------------------------------------------------------ launch

// TMA boxes serve a block size that is a multiple of 8 dividing 128 (each box
// lands on whole 1024-byte swizzle groups); other sizes are gathered.
static bool boxes(int bs) { return bs % 8 == 0 && TK % bs == 0; }

// q [T][H][d]: box = 64 columns x `heads` heads x tpt tokens.
static bool make_tmap_q(CUtensorMap* map, const void* q, int T, int H, int d, int heads, int tpt) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tpt};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int LOAD, bool CHUNKS>
static cudaError_t launch(const Extend& p, const void* q, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  if (!make_tmap_q(&tq, q, p.T, p.H, D, p.heads, p.tpt)) return cudaErrorInvalidValue;
  if (LOAD == BOXES) {
    if (!make_tmap_bf16(&tk, p.k_cache, p.num_blocks * p.Hkv, p.bs, D, p.bs) ||
        !make_tmap_bf16(&tv, p.v_cache, p.num_blocks * p.Hkv, p.bs, D, p.bs))
      return cudaErrorInvalidValue;
  } else {
    tk = tv = tq;  // unused
  }
  auto kern = extend_kernel<D, LOAD, CHUNKS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, LOAD>::ALLOC);
  if (e != cudaSuccess) return e;
  kern<<<p.ctas, Threads<LOAD>::N, Smem<D, LOAD>::ALLOC, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  const int jobs = p.ctas - 1 + p.n_long;
  if (e != cudaSuccess || jobs == 0) return e;  // one CTA: nothing is cut
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(jobs));
  cfg.blockDim = dim3(MERGE_THREADS);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, extend_merge_kernel<D, CHUNKS>, p);
}

}  // namespace ext

size_t extend_sizes(Extend* p, int d, bool q4) {
  using namespace ext;
  p->bs_inverse = static_cast<unsigned>((1ull << 32) / p->bs + 1);
  const int G = p->H / p->Hkv, parts = (G + BM - 1) / BM;
  p->heads = (G + parts - 1) / parts;
  p->hv = p->Hkv * parts;
  p->tpt = BM / p->heads;
  const long long span = 2 * p->tpt;
  const long long ctx = static_cast<long long>(p->max_blocks) * p->bs;
  // A chunk's K and V, of all K/V heads, stay in L2 (read as they lie there).
  const long long key_bytes = 2ll * p->Hkv * (q4 ? d / 2 + d / 16 : 2 * d);
  const long long lc = kL2GroupBytes / key_bytes / TK * TK;
  p->lc = static_cast<int>(lc < 8 * TK ? 8 * TK : lc > (1 << 29) ? 1 << 29 : lc);
  const long long items = p->hv * (p->T / span + (p->T < p->B ? p->T : p->B));  // at most
  const long long shares = items * (ctx + PIECE) / MIN_SHARE;
  p->ctas = static_cast<int>(shares < 1 ? 1 : shares > MAX_CTAS ? MAX_CTAS : shares);
  p->chunk_halves = d == 128 && !q4 ? CHUNK_HALVES_512 : CHUNK_HALVES;
  p->may_chunk = p->T > (CHUNK_ITEMS - 1) * span && ctx > p->lc;
  p->n_long = 0;
  long long whole = 0;
  if (p->may_chunk) {
    // Items of requests with two or more: at most 2 T / span. A chunk is at
    // least a share long, and a long item passes at most twice its keys / lc.
    const long long long_items = p->hv * (2ll * p->T / span), by_share = 2ll * p->ctas;
    p->n_long = static_cast<int>(long_items < by_share ? long_items : by_share);
    whole = long_items * ((ctx + p->lc - 1) / p->lc);
    if (whole > by_share) whole = by_share;
  }
  p->n_slots = static_cast<int>(2 * p->ctas + whole);
  return static_cast<size_t>(p->n_slots) * ROWS * (d + 1) * sizeof(float) + p->ctas * sizeof(ItemCut);
}

cudaError_t launch_extend(const Extend& p, const void* q, int d, bool q4, cudaStream_t stream) {
  using namespace ext;
  auto go = [&](auto chunks) {
    constexpr bool C = decltype(chunks)::value;
    if (q4) return d == 64 ? launch<64, CODES, C>(p, q, stream) : launch<128, CODES, C>(p, q, stream);
    if (boxes(p.bs)) return d == 64 ? launch<64, BOXES, C>(p, q, stream) : launch<128, BOXES, C>(p, q, stream);
    return d == 64 ? launch<64, GATHER, C>(p, q, stream) : launch<128, GATHER, C>(p, q, stream);
  };
  return p.may_chunk ? go(std::true_type{}) : go(std::false_type{});
}

cudaError_t read_and_clear_extend_error(uint32_t* out, cudaStream_t stream) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_extend_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbolAsync(g_extend_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return e;
  return cudaStreamSynchronize(stream);
}

}  // namespace fa
