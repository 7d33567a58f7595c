// Decode attention against a paged KV cache held in 4-bit codes (fa_q4.cuh
// has the codes; fa_decode.cu the same step over a bf16 cache, the context
// split and the merge of the splits' results).
//
// A cached value is z + s (n − 8), with one (s, z) per group of 64
// dimensions, so with the groups' partial products
//     q·k = Σ_groups s (Σ_c q_c (n_c − 8)) + z Σ_c q_c,
//     o   = Σ_keys (p s) (n − 8) + Σ_keys p z,
// and both products of a tile run on the tensor core over the codes
// themselves, which bf16 holds exactly; steps and centres are applied to the
// score accumulators and to the probabilities, in fp32.
//
// The step would be bound by reading the codes, d/2 + d/16 bytes a key or
// value: at 6.8 TB/s an SM takes in 21 bytes a clock, 38 values, and each has
// to be turned into an operand. tcgen05 takes operands from shared memory or
// TMEM, and writing 38 bf16 values a clock to shared memory and reading them
// back, 153 bytes, is more than its 128 bytes a clock (one-byte operands, a
// code as e4m3's n 2^-9, would be 77; not built). So a warp keeps them in
// registers: mma.sync m16n8k16, whose A operand is 16 keys (scores) or 16 dimensions
// (output) and whose 8 columns are query heads that share the K/V head.
//   scores  Sᵀ[key][head]: rows g and g + 8 of a tile are keys; the words of
//           a key's row go to the lane quarter t that needs them as they are
//           (the order of the products' inner index is free: q is read in
//           the same order).
//   output  Oᵀ[dim][head]: an operand register pairs two keys of one
//           dimension, two words' halves merged by one byte permutation.
// A nibble becomes a bf16 number by placing it in the top four mantissa bits
// of 16.0 (16 + n: one shift, one and-or for two values), or an fp16 one in
// the low bits of 1024. Keys have the offset subtracted; the values' offsets
// cancel between the halves of a stage.
//
// What bounds it, measured (32 requests of 2k to 8k tokens, 8 K/V heads, d =
// 128, 189 MB): 70 us with the merge. A stage of 32 keys costs a warp about
// 690 instructions, nearly half of them on the integer pipe at two clocks
// each, and 36 mma.sync at 8 clocks of the tensor pipe each. No pipe is full
// (integer 52%, tensor 19%, DRAM 38%): at 12 warps an SM the latencies between
// dependent steps keep the schedulers to 46% of their issue slots. Before
// probabilities went in as two numbers (below) the step took 69 us, and where
// one cache is read again and again 65; of those the copies alone took 37 and
// the products alone, on whatever the ring holds, 53. At that time 12, 16 or
// 20 warps an SM, 16-key steps and scores one tile ahead of the output all
// measured within 5%, or slower; so did 8-bit products over the nibbles as they
// are (a byte n is e4m3's n 2^-9), which the compiler expands into conversions
// and 16-bit products: 77 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_ptx.cuh"

namespace fa {

static __device__ uint32_t g_decq4_err;

namespace decq4 {

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int TK = 32;          // keys a warp takes of a tile
constexpr int CK = WARPS * TK;  // keys of a CTA's tile: one stage of the ring
constexpr float LN2 = 0.69314718055994531f;
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t NO_ROW = 0xffffffffu;  // the host keeps the cache below 2^32 - 1 rows

// A stage of the ring holds a tile: K codes, V codes, K pairs, V pairs of its
// 128 keys, 32 for each warp. Three CTAs an SM at d = 128 (160 registers a
// thread; four at 128 registers measured the same, with more instructions),
// four at d = 64, two with 16 query heads a CTA.
template <int D, int NT>
struct Ring {
  static constexpr int CTAS = NT == 1 ? (D == 64 ? 4 : 3) : 2;  // per SM
  static constexpr int CODES = CK * D / 2, PAIRS = CK * D / 16;
  static constexpr int KC = 0, VC = CODES, KS = 2 * CODES, VS = KS + PAIRS;
  static constexpr int STAGE = 2 * CODES + 2 * PAIRS;
  static constexpr int STAGES = (D == 64 ? 6 : 3) + (CTAS == 3);
  static constexpr int BAR_OFF = STAGES * STAGE;  // full [STAGES] (GATHER: [WARPS][STAGES]), empty [STAGES]
  static constexpr int MASK_OFF = BAR_OFF + (WARPS + 1) * STAGES * 8;  // [STAGES][WARPS] keys that are there
  static constexpr int BYTES = MASK_OFF + STAGES * WARPS * 4;
  static_assert(CTAS * (BYTES + 1024) <= 233472, "the CTAs must fit an SM");
  // at the end the ring takes the warps' results: [8 NT heads][D + 1], m and
  // l [8 NT], and the weights [8 NT][WARPS], fp32
  static constexpr int RESULT = 8 * NT * (D + 1 + 2 + WARPS) * 4;
  static_assert(WARPS * RESULT <= STAGES * STAGE, "the ring holds the warps' results");
};

// d (+)= A (16x16) B (16x8), fp32; both operands fp16, or both bf16.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// (v & mask) | base in one instruction. The bases come in as kernel
// arguments: as constants beside a constant mask they would take a second
// instruction each.
struct Bases {
  uint32_t key, value;  // two fp16 1024, two bf16 16
};
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t base) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "r"(mask), "r"(base));
  return d;
}

__device__ __forceinline__ uint32_t andnot_or(uint32_t v, uint32_t mask, uint32_t base) {  // (~v & mask) | base
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xae;" : "=r"(d) : "r"(v), "r"(mask), "r"(base));
  return d;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Keys: the four nibbles of each 16-bit half as four pairs of fp16: n − 8
// (nibbles 0 and 2, in the lowest mantissa bits of 1024, less 1032) and
// 16 (n − 8) (nibbles 1 and 3, four bits up, less 16 · 72), both exact: one
// shift, four and-ors and four subtractions (on the other pipe) for 8 values.
// Left in the operands, the offsets would be taken off a score at the end,
// and what fp32 loses beside 1024 Σ q is 3e-5 of a score.
__device__ __forceinline__ void key_pairs(uint32_t w, uint32_t base, uint32_t (&v)[4]) {
  const uint32_t h = w >> 8;
  v[0] = sub_f16x2(and_or(w, 0x000f000fu, base), 0x64086408u);
  v[1] = sub_f16x2(and_or(w, 0x00f000f0u, base), 0x64806480u);
  v[2] = sub_f16x2(and_or(h, 0x000f000fu, base), 0x64086408u);
  v[3] = sub_f16x2(and_or(h, 0x00f000f0u, base), 0x64806480u);
}
// Values: 16 + n for nibble I of each half, as two bf16 (n in the top four
// mantissa bits of 16), or 16 + 15 − n with FLIP (the complement's bits).
template <int I, bool FLIP>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, uint32_t base) {
  const uint32_t v = I == 0 ? w << 3 : w >> (4 * I - 3);
  return FLIP ? andnot_or(v, 0x00780078u, base) : and_or(v, 0x00780078u, base);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Contiguous copy global -> shared by the copy engine, completing bytes on
// the mbarrier: addresses and size are multiples of 16.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// 4- or 8-byte asynchronous copy global -> shared.
template <int N>
__device__ __forceinline__ void cp_async_small(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(__cvta_generic_to_global(src)),
               "n"(N)
               : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// x / n for x < 2^30 and a fixed n, by a product with ceil(2^(30 + k) / n),
// 2^(k-1) < n <= 2^k: the multiplier is off by less than n 2^-k <= 1 in units
// of 2^-30 / n, too little to carry any x < 2^30 past the next integer.
struct Divide {
  uint32_t mul, shift;
  static Divide of(int n) {
    int k = 0;
    while ((1ll << k) < n) ++k;
    return {static_cast<uint32_t>(((1ull << (30 + k)) + n - 1) / n), static_cast<uint32_t>(30 + k)};
  }
  __device__ __forceinline__ int operator()(int x) const {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(x)) * mul) >> shift);
  }
};

// How a stage is filled. BULK (a block size with a factor of 8): runs of
// `run` = 8 .. 128 consecutive slots of one block are contiguous, and a lane
// copies one run of codes or pairs in one piece; the warps take turns to fill
// whole tiles, so the bookkeeping of a tile is done once for all four.
// GATHER (any other): a lane looks up one key's row and the rows go over in
// 16-byte pieces, each warp filling its own part of the tile.
enum Fill : int { BULK = 0, GATHER = 1 };

// One CTA: split s of request b's context, K/V head hk, NH query heads in
// 8·NT columns of the products.
//
// A probability times a value's step, p s, goes into the output product as
// two bf16 numbers, its rounding and what that leaves: 2^-16 of it is lost
// (of one bf16 number 2^-8, by which the output was 1.35 times as far from 64
// bits as its own rounding). With up to four query heads a K/V head (FOLD)
// half of the columns would be empty: columns 4 .. 7 are the same heads again
// and take the second part, so the products stay as many (the 32 requests of
// the file's head: 69.4 us with one number, 70.2 so; two contexts of 100k and
// 131k tokens 70.4 and 72.3). More heads take a second product for it (75 and
// 80 us in those two cases; 16 requests of 1k to 8k tokens, one-token blocks,
// 16 heads a K/V head: 24.8 us with one number, 28.6 so).
template <int D, int NT, bool FOLD, int FILL>
__global__ void __launch_bounds__(THREADS, (Ring<D, NT>::CTAS))
    decode_q4_kernel(const DecodeQ4 p, int run, Divide by_bs, Bases bases) {
  using R = Ring<D, NT>;
  constexpr int NG = D / 64;    // groups of a row
  constexpr int NC = 8 * NT;    // columns
  constexpr int NH = FOLD ? 4 : NC;  // query heads of the CTA
  constexpr int MT = D / 16;    // 16-dimension tiles of the output
  constexpr int ST = R::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* err = &g_decq4_err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int S = gridDim.x, s = blockIdx.x, b = blockIdx.z;
  const int G_all = p.H / p.Hkv, n_chunk = (G_all + NH - 1) / NH;
  const int hk = blockIdx.y / n_chunk, chunk = blockIdx.y % n_chunk;
  const int G = min(NH, G_all - NH * chunk);
  const int head0 = b * p.H + hk * G_all + NH * chunk;
  const long long prow = static_cast<long long>(s) * p.B * p.H + head0;
  const long long part_rows = static_cast<long long>(S) * p.B * p.H;

  int L = in_range(b, 1, p.B, err) ? p.seq_lens[b] : 0;
  L = L < 0 ? 0 : (L > p.max_blocks * p.bs ? p.max_blocks * p.bs : L);
  const int n_tiles = (L + CK - 1) / CK;
  const int tps = (n_tiles + S - 1) / S;
  const int tile0 = s * tps;
  const int n = max(0, min(n_tiles, tile0 + tps) - tile0);  // this CTA's tiles

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R::BAR_OFF) + (FILL == BULK ? 0 : warp * ST);
  uint64_t* empty = reinterpret_cast<uint64_t*>(smem + R::BAR_OFF) + WARPS * ST;  // BULK
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + R::MASK_OFF);
  if (FILL == BULK) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < ST; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], WARPS);
      }
      fence_mbar_init();
    }
    __syncthreads();
  } else {
    if (lane == 0) {
      for (int i = 0; i < ST; ++i) mbar_init(&full[i], 32);
      fence_mbar_init();
    }
    __syncwarp();
  }

  // A lane's lookups for a tile. BULK: copy lane + 32 i of the tile's
  // 4 · 128 / run, part (lane & 3) of a run; the run's first token. GATHER:
  // the warp's key `lane`.
  constexpr int LOOK = FILL == BULK ? 2 : 1;
  const long long rows = static_cast<long long>(p.num_blocks) * p.Hkv * p.bs;
  auto token_of = [&](int j, int i) {
    return (tile0 + j) * CK + (FILL == BULK ? ((lane + 32 * i) >> 2) * run : warp * TK + lane);
  };
  auto there = [&](int j, int i) {
    return j < n && token_of(j, i) < L && (FILL == GATHER || ((lane + 32 * i) >> 2) * run < CK);
  };
  struct Entries {
    int e[LOOK];
  };
  auto look = [&](int j) {  // the table's entries
    Entries x;
#pragma unroll
    for (int i = 0; i < LOOK; ++i) {
      x.e[i] = -1;
      if (there(j, i)) {
        const long long ti = static_cast<long long>(b) * p.max_blocks + by_bs(token_of(j, i));
        if (in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err)) x.e[i] = p.block_table[ti];
      }
    }
    return x;
  };
  auto row_of = [&](int tok, int entry) {
    return (static_cast<uint32_t>(entry) * p.Hkv + hk) * static_cast<uint32_t>(p.bs) +
           static_cast<uint32_t>(tok - by_bs(tok) * p.bs);
  };
  // Fill stage st with tile j (the warp's part of it), run by a whole warp.
  auto fill = [&](int j, int st, const Entries& x) {
    uint8_t* stage = smem + st * R::STAGE;
    if constexpr (FILL == BULK) {
      // parts: 0 K codes, 1 V codes, 2 K pairs, 3 V pairs
      const int part = lane & 3;
      const int per_key = part < 2 ? D / 2 : D / 16;
      const uint8_t* base = part == 0 ? p.k_cache : part == 1 ? p.v_cache
                            : reinterpret_cast<const uint8_t*>(part == 2 ? p.k_scale : p.v_scale);
      uint8_t* dst = stage + (part == 0 ? R::KC : part == 1 ? R::VC : part == 2 ? R::KS : R::VS);
      const uint32_t bytes = run * per_key;
      uint32_t row[LOOK], mine = 0;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < LOOK; ++i) {
        row[i] = NO_ROW;
        if (!there(j, i)) continue;
        if (x.e[i] >= 0 && x.e[i] < p.num_blocks) row[i] = row_of(token_of(j, i), x.e[i]);
        else bad = true;
        if (row[i] != NO_ROW &&
            !in_range(static_cast<long long>(row[i]) * per_key, bytes, rows * per_key, err))
          row[i] = NO_ROW;
        if (row[i] != NO_ROW) mine += bytes;
      }
      const uint32_t total = __reduce_add_sync(0xffffffffu, mine);
      uint32_t present = 0xffffffffu;      // in lane w < WARPS: warp w's keys
      if (__any_sync(0xffffffffu, bad)) {  // blocks outside the cache: their keys are skipped
        if (bad) atomicExch(err, DEV_BAD_INDEX);
        for (int w = 0; w < WARPS; ++w) {
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < LOOK; ++i) {
            const int k0 = ((lane + 32 * i) >> 2) * run - 32 * w;  // the run's first key in this word
            if (part == 0 && row[i] != NO_ROW)
              for (int k = max(k0, 0); k < min(k0 + run, 32); ++k) bits |= 1u << k;
          }
          bits = __reduce_or_sync(0xffffffffu, bits);
          if (lane == w) present = bits;
        }
      }
      if (lane < WARPS) masks[st * WARPS + lane] = present;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[st], total);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < LOOK; ++i)
        if (row[i] != NO_ROW)
          bulk_load(dst + ((lane + 32 * i) >> 2) * bytes, base + static_cast<size_t>(row[i]) * per_key, bytes, &full[st]);
    } else {
      constexpr int CH = D / 32;     // 16-byte chunks of a row of codes
      constexpr int RPI = 32 / CH;   // rows per warp instruction
      const bool in = there(j, 0), live = in && x.e[0] >= 0 && x.e[0] < p.num_blocks;
      if (in && !live) atomicExch(err, DEV_BAD_INDEX);
      const uint32_t row = live ? row_of(token_of(j, 0), x.e[0]) : NO_ROW;
      const uint32_t mask = __ballot_sync(0xffffffffu, live);
      if (lane == 0) masks[st * WARPS + warp] = mask;
      uint8_t* kc = stage + R::KC + warp * TK * (D / 2);
      uint8_t* vc = stage + R::VC + warp * TK * (D / 2);
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int key = i * RPI + lane / CH;
        const uint32_t rw = __shfl_sync(0xffffffffu, row, key);
        const size_t off = static_cast<size_t>(rw) * (D / 2) + c * 16;
        if (rw != NO_ROW && in_range(off, 16, rows * (D / 2), err)) {
          cp_async_16(kc + key * (D / 2) + c * 16, p.k_cache + off, 16);
          cp_async_16(vc + key * (D / 2) + c * 16, p.v_cache + off, 16);
        }
      }
      const size_t so = static_cast<size_t>(row) * NG;
      if (live && in_range(so, NG, rows * NG, err)) {
        cp_async_small<NG * 4>(stage + R::KS + (warp * TK + lane) * (NG * 4), p.k_scale + so);
        cp_async_small<NG * 4>(stage + R::VS + (warp * TK + lane) * (NG * 4), p.v_scale + so);
      }
      cp_async_arrive_noinc(&full[st]);
    }
  };
  // The first ST tiles: BULK, warp i mod 4 fills tile i; GATHER, all of them.
  // `next` is the tile this warp fills next, with its entries in `ahead`.
  int next;
  Entries ahead;
  if (FILL == BULK) {
    for (int i = warp; i < min(ST, n); i += WARPS) fill(i, i, look(i));
    next = ST + (warp + WARPS - 1) % WARPS;  // by turn: at the end of tile j warp j mod 4 fills j - 1 + ST
    ahead = look(next);
  } else {
    Entries first[ST];
#pragma unroll
    for (int i = 0; i < ST; ++i) first[i] = look(i);
#pragma unroll
    for (int i = 0; i < ST; ++i)
      if (i < n) fill(i, i, first[i]);
    next = ST;
    ahead = look(next);
  }

  // Query operand: for group gr and word w of a lane quarter's 16 dimensions
  // 64 gr + 16 t + 8 w + 0..7, K step 2 w + h (h = 0, 1) multiplies elements
  // (2h, 2h + 4), whose codes come as n − 8, and (2h + 1, 2h + 5), whose come
  // as 16 (n − 8): the latter's q carry the 1/16. A head's q are scaled by a
  // power of two to a largest magnitude in [1, 2): fp16 then holds elements
  // down to 2^-13 of that (those without the 1/16: 2^-17) exactly, and smaller
  // ones to within 2^-21 (2^-25) of it.
  uint32_t qf[NT][NG][4][2];
  float qsum[NT][NG][2];  // Σ q of this lane's columns 2t, 2t + 1
  float sc[NT][2];        // score units to log2 units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint4 v[NG][2];
    float top = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        v[gr][w] = make_uint4(0, 0, 0, 0);
        const int h = FOLD ? g % NH : nt * 8 + g;
        const long long off = static_cast<long long>(head0 + h) * D + gr * 64 + t * 16 + w * 8;
        if (h < G && in_range(off, 8, static_cast<long long>(p.B) * p.H * D, err))
          v[gr][w] = *reinterpret_cast<const uint4*>(p.q + off);
        const uint32_t u[4] = {v[gr][w].x, v[gr][w].y, v[gr][w].z, v[gr][w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf_lo(u[i])), fabsf(bf_hi(u[i]))));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^-e with 2^e <= top < 2^(e+1), kept within the normal range
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = e < -126 ? -126 : e > 126 ? 126 : e;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    // of column g; never 0 (at least the smallest fp32 number), or a masked
    // score's -inf would become NaN
    const float up = fmaxf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2, __uint_as_float(1u));
    sc[nt][0] = __shfl_sync(0xffffffffu, up, 8 * t);      // lanes of column 2t
    sc[nt][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);  // and of column 2t + 1
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 x = v[gr][w];  // elements (0, 1), (2, 3), (4, 5), (6, 7)
        const float d16 = down * 0.0625f;
        qf[nt][gr][2 * w][0] = pack_f16x2(bf_lo(x.x) * down, bf_lo(x.z) * down);
        qf[nt][gr][2 * w][1] = pack_f16x2(bf_hi(x.x) * d16, bf_hi(x.z) * d16);
        qf[nt][gr][2 * w + 1][0] = pack_f16x2(bf_lo(x.y) * down, bf_lo(x.w) * down);
        qf[nt][gr][2 * w + 1][1] = pack_f16x2(bf_hi(x.y) * d16, bf_hi(x.w) * d16);
      }
      // Σ q of what fp16 holds: a product with constants. Registers 2 and 3
      // of A meet the second half of a K step.
      const uint32_t one = 0x3c003c00u, x16 = 0x4c004c00u;  // 1, 16
      const uint32_t ones[4] = {one, one, x16, x16};
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma_f16(c, ones, qf[nt][gr][ks][0], qf[nt][gr][ks][1]);
      qsum[nt][gr][0] = c[0], qsum[nt][gr][1] = c[1];
    }
  }

  // Output sums. The first 16 keys of a stage add p s (16 + n), the others
  // −p s (31 − n): the offsets of the two nearly cancel, so the running sums
  // stay as small as those of n − 8 and lose no more (the tensor core cuts
  // sums off at 24 bits). `fix` takes Σ ∓24, 23 p s of the same rounded p s,
  // what is left between the offsets and −8: one product for a group's four.
  float acc[NT][MT][4], fix[NT][NG][4];
  // Per column: the exponents' reference in log2 units (0 while no key has been
  // seen), the score above which it is raised, and the running sums.
  float m[NT][2], lim[NT][2], l[NT][2], zc[NT][NG][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int e = 0; e < 4; ++e) fix[nt][gr][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = 0.f;
      lim[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) zc[nt][gr][e] = 0.f;
    }
  }

  // FOLD: the bytes of a pair's rounded numbers that are taken off its own
  // (none in the columns of the first part), as fp32.
  const uint32_t off_lo = FOLD && t < 2 ? 0x4444u : 0x1044u, off_hi = FOLD && t < 2 ? 0x4444u : 0x3244u;

  bool ok = true;
  int st = 0, stop = n;
  uint32_t phase = 0;
  for (int j = 0; j < stop; ++j, phase ^= st + 1 == ST, st = st + 1 == ST ? 0 : st + 1) {
    if (!mbar_wait_warp(&full[st], phase, err) && ok) {
      ok = false;
      stop = min(n, j + ST);  // wait for what is in flight, fill no more
    }
    if (!ok) continue;
    __syncwarp();  // the mask
    const int left = L - (tile0 + j) * CK - warp * TK;
    uint32_t mask = masks[st * WARPS + warp];
    if (left < TK) mask &= left > 0 ? (1u << left) - 1u : 0u;
    const uint8_t* stage = smem + st * R::STAGE;
    const uint8_t* kc = stage + R::KC + warp * TK * (D / 2);
    const uint8_t* vc = stage + R::VC + warp * TK * (D / 2);
    const uint8_t* kps = stage + R::KS + warp * TK * (D / 16);
    const uint8_t* vps = stage + R::VS + warp * TK * (D / 16);

    // Scores: x[nt][u][2 r + e] is key 16 u + g + 8 r, column 2 t + e.
    float x[NT][2][4];
    uint32_t vp[2][2][NG];  // the keys' value pairs
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t kp[2][NG];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = 16 * u + g + 8 * r;
        if (NG == 2) {
          const uint2 a = *reinterpret_cast<const uint2*>(kps + key * 8);
          const uint2 c = *reinterpret_cast<const uint2*>(vps + key * 8);
          kp[r][0] = a.x, kp[r][NG - 1] = a.y, vp[u][r][0] = c.x, vp[u][r][NG - 1] = c.y;
        } else {
          kp[r][0] = *reinterpret_cast<const uint32_t*>(kps + key * 4);
          vp[u][r][0] = *reinterpret_cast<const uint32_t*>(vps + key * 4);
        }
      }
      uint32_t a[NG][4][4];  // per K step
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = 16 * u + g + 8 * r;
          const uint2 w = *reinterpret_cast<const uint2*>(kc + key * (D / 2) + gr * 32 + t * 8);
          uint32_t v[4];
          key_pairs(w.x, bases.key, v);
          a[gr][0][r] = v[0], a[gr][0][r + 2] = v[1], a[gr][1][r] = v[2], a[gr][1][r + 2] = v[3];
          key_pairs(w.y, bases.key, v);
          a[gr][2][r] = v[0], a[gr][2][r + 2] = v[1], a[gr][3][r] = v[2], a[gr][3][r + 2] = v[3];
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[NG][4] = {};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) mma_f16(c[gr], a[gr][ks], qf[nt][gr][ks][0], qf[nt][gr][ks][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = bf_hi(kp[e >> 1][0]) * qsum[nt][0][e & 1];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            if (gr > 0) v = fmaf(bf_hi(kp[e >> 1][gr]), qsum[nt][gr][e & 1], v);
            v = fmaf(bf_lo(kp[e >> 1][gr]), c[gr][e], v);
          }
          x[nt][u][e] = v;
        }
      }
    }
    if (mask != 0xffffffffu) {
      // Dead keys: their codes are finite whatever the slot holds, their
      // pairs need not be.
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool dead = ((mask >> (16 * u + g + 8 * r)) & 1u) == 0;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) vp[u][r][gr] = dead ? 0u : vp[u][r][gr];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            x[nt][u][2 * r] = dead ? -INFINITY : x[nt][u][2 * r];
            x[nt][u][2 * r + 1] = dead ? -INFINITY : x[nt][u][2 * r + 1];
          }
        }
    }
    bool need = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        need |= fmaxf(fmaxf(x[nt][0][e], x[nt][0][e + 2]), fmaxf(x[nt][1][e], x[nt][1][e + 2])) > lim[nt][e];
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(fmaxf(x[nt][0][e], x[nt][0][e + 2]), fmaxf(x[nt][1][e], x[nt][1][e + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          v *= sc[nt][e];
          if (v == -INFINITY) continue;  // no key of this head yet, nothing to scale
          const bool first = lim[nt][e] == -INFINITY;
          const float m_new = first ? v : fmaxf(m[nt][e], v);
          const float alpha = first ? 0.f : ex2(m[nt][e] - m_new);
          m[nt][e] = m_new;
          lim[nt][e] = (m_new + RESCALE_LOG2) / sc[nt][e];
          l[nt][e] *= alpha;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            zc[nt][gr][e] *= alpha;
            fix[nt][gr][e] *= alpha;  // (rows are alike: the first is read at the end)
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[nt][i][e] *= alpha;
            acc[nt][i][e + 2] *= alpha;
          }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // Probabilities, times the values' steps, as the output's B operand.
      uint32_t pf[NT][NG][2], pf2[NT][NG][2];  // pf2: the second parts of all heads, not FOLD
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = ex2(fmaf(x[nt][u][e], sc[nt][e & 1], -m[nt][e & 1]));  // a dead key's -inf gives 0
          l[nt][e & 1] += pr[e];
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float sv = u == 0 ? bf_lo(vp[u][r][gr]) : -bf_lo(vp[u][r][gr]), zv = bf_hi(vp[u][r][gr]);
            zc[nt][gr][0] = fmaf(pr[2 * r], zv, zc[nt][gr][0]);
            zc[nt][gr][1] = fmaf(pr[2 * r + 1], zv, zc[nt][gr][1]);
            // (bf16 for its range: fp16 would need a reference of its own for
            // the steps. A step times p <= 2^8 has to stay finite.)
            const float p0 = pr[2 * r] * sv, p1 = pr[2 * r + 1] * sv;
            const uint32_t rounded = pack_bf16x2(p0, p1);
            const uint32_t left = pack_bf16x2(p0 - __uint_as_float(__byte_perm(rounded, 0u, off_lo)),
                                              p1 - __uint_as_float(__byte_perm(rounded, 0u, off_hi)));
            pf[nt][gr][r] = transpose8x8(FOLD ? left : rounded);
            if (!FOLD) pf2[nt][gr][r] = transpose8x8(left);
          }
      }
      // Output: tile 4 gr + i has dimension 64 gr + 8 g + i in row g, + 4 in row g + 8.
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          w[r] = *reinterpret_cast<const uint32_t*>(vc + (16 * u + 2 * t + (r & 1) + 8 * (r >> 1)) * (D / 2) +
                                                    gr * 32 + g * 4);
        const uint32_t h[4] = {__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                               __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632)};
        uint32_t a[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (u == 0) {
            a[0][r] = value_pair<0, false>(h[r], bases.value), a[1][r] = value_pair<1, false>(h[r], bases.value);
            a[2][r] = value_pair<2, false>(h[r], bases.value), a[3][r] = value_pair<3, false>(h[r], bases.value);
          } else {
            a[0][r] = value_pair<0, true>(h[r], bases.value), a[1][r] = value_pair<1, true>(h[r], bases.value);
            a[2][r] = value_pair<2, true>(h[r], bases.value), a[3][r] = value_pair<3, true>(h[r], bases.value);
          }
        }
        // -24, and 23 of a negated probability
        const uint32_t c = u == 0 ? 0xc1c0c1c0u : 0xc1b8c1b8u;
        const uint32_t off[4] = {c, c, c, c};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          auto products = [&](const uint32_t (&b)[2]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[nt][4 * gr + i], a[i], b[0], b[1]);
            mma_bf16(fix[nt][gr], off, b[0], b[1]);
          };
          products(pf[nt][gr]);
          if (!FOLD) products(pf2[nt][gr]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (FILL == BULK) {
      if (lane == 0) mbar_arrive(&empty[st]);
      // The turn's warp fills the stage before this one, which every warp left
      // a tile ago or is about to.
      if (j % WARPS == warp && j > 0) {
        const int before = st == 0 ? ST - 1 : st - 1;
        if (next < n) {
          if (mbar_wait_warp(&empty[before], st == 0 ? phase ^ 1 : phase, err)) {
            fill(next, before, ahead);
          } else {
            ok = false;
            stop = min(n, j + ST);
          }
        }
        next += WARPS;
        ahead = look(next);
      }
    } else if (next < n) {
      fill(next, st, ahead);
      ahead = look(++next);
    }
  }

  // The warps' results: Σ over the lanes that hold other keys, then one
  // (m, l, o) per column and warp, in the ring (every copy has landed and been
  // read).
  constexpr int OROW = D + 1;
  auto sm_o = [&](int w) { return reinterpret_cast<float*>(smem + w * R::RESULT); };
  auto sm_m = [&](int w) { return sm_o(w) + NC * OROW; };
  auto sm_l = [&](int w) { return sm_m(w) + NC; };
  if (FILL == GATHER) {  // nothing may land after this
    cp_async_commit();
    cp_async_wait<0>();
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = nt * 8 + 2 * t + e;
      float lv = l[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lv += __shfl_xor_sync(0xffffffffu, lv, o);
      if (g == 0) {
        sm_m(warp)[col] = m[nt][e];
        sm_l(warp)[col] = lv;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float z = zc[nt][gr][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        z = (FOLD && t >= 2 ? 0.f : z) + fix[nt][gr][e];  // a head's centres count once
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = col * OROW + 64 * gr + 8 * g + i;
          if (!in_range(at, 5, NC * OROW, err)) continue;
          sm_o(warp)[at] = acc[nt][4 * gr + i][e] + z;
          sm_o(warp)[at + 4] = acc[nt][4 * gr + i][e + 2] + z;
        }
      }
    }
  __syncthreads();
  // One lane per head: the warps' weights e^(m_w − m) / Σ, behind the first
  // warp's result; then every thread sums a column of some heads.
  float* weights = sm_m(0) + 2 * NC;  // [NH][WARPS]
  if (threadIdx.x < G) {
    const int h = threadIdx.x;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (sm_l(w)[h] != 0.f) mm = fmaxf(mm, sm_m(w)[h]);
    float a[WARPS], lt = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      // l = 0: a warp that saw no key (and o = 0). A NaN score leaves l NaN,
      // and the head's result with it.
      a[w] = sm_l(w)[h] == 0.f ? 0.f : ex2(sm_m(w)[h] - mm);
      lt = fmaf(a[w], sm_l(w)[h], lt);
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) weights[h * WARPS + w] = a[w] * inv;
    if (in_range(prow + h, 1, part_rows, err))
      (S == 1 ? p.lse : p.lse_part)[prow + h] = lt == 0.f ? -INFINITY : (mm + __log2f(lt)) * LN2;
  }
  __syncthreads();
  const int c = threadIdx.x % D;
  for (int h = threadIdx.x / D; h < G; h += THREADS / D) {
    float ov = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float* o = sm_o(w) + h * OROW + c;
      ov = fmaf(weights[h * WARPS + w], FOLD ? o[0] + o[NH * OROW] : o[0], ov);
    }
    const long long at = (prow + h) * D + c;
    if (in_range(at, 1, part_rows * D, err)) {
      if (S == 1) p.o[at] = __float2bfloat16_rn(ov);
      else p.o_part[at] = ov;
    }
  }
}

template <int D, int NT, bool FOLD, int FILL>
static cudaError_t launch_f(const DecodeQ4& p, int S, int run, cudaStream_t stream) {
  auto kern = decode_q4_kernel<D, NT, FOLD, FILL>;
  const int smem = Ring<D, NT>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int n_chunk = (p.H / p.Hkv + 8 * NT - 1) / (8 * NT);
  const dim3 grid(static_cast<unsigned>(S), static_cast<unsigned>(p.Hkv * n_chunk), static_cast<unsigned>(p.B));
  kern<<<grid, THREADS, smem, stream>>>(p, run, Divide::of(p.bs), Bases{0x64006400u, 0x41804180u});
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch(const DecodeQ4& p, int S, cudaStream_t stream) {
  int run = p.bs & -p.bs;  // slots of a block from a multiple of this on are contiguous for as many keys
  if (run > CK) run = CK;
  const bool bulk = run >= 8;
  const int G = p.H / p.Hkv;
  if (G <= 4) return bulk ? launch_f<D, 1, true, BULK>(p, S, run, stream) : launch_f<D, 1, true, GATHER>(p, S, run, stream);
  if (G <= 8) return bulk ? launch_f<D, 1, false, BULK>(p, S, run, stream) : launch_f<D, 1, false, GATHER>(p, S, run, stream);
  return bulk ? launch_f<D, 2, false, BULK>(p, S, run, stream) : launch_f<D, 2, false, GATHER>(p, S, run, stream);
}

}  // namespace decq4

// Splits that fill the GPU. CTAs come three (with more than eight query heads a
// K/V head two) to an SM; the rule takes one wave of them for one or two
// requests and three waves for more, whose lengths the host does not know, and
// no split below 1024 keys. GPU time in us by splits, the rule's in brackets:
//     32 requests of 2k to 8k tokens, 8 K/V heads   2: 80   [5: 71]  10: 74  15: 79
//     16 of 1k to 8k, 2 K/V heads of 16 heads       4: 38   [8: 29]  10: 27  16: 31
//     1 of 131k, 8 K/V heads                        28: 68  [57: 55] 85: 74  114: 71
//     2 of 100k and 131k                            14: 98  [28: 72] 42: 91  56: 82
//     2 of 1k and 131k                              14: 97  [28: 72] 42: 68  56: 60
//     3 of 87k                                      28: 106 [57: 99] 85: 112
//     3 of 1k to 131k                               28: 80  [57: 80] 85: 90
//     4 of 16k, 2 K/V heads                         8: 27   [16: 20] 32: 18  64: 25
//     1 of 8k, 1 K/V head                           4: 27   [8: 19]  16: 14  32: 14
//     3 of up to 700, 12 K/V heads, d = 64          [1: 12.3] 2: 11.7  3: 11.6  6: 10.3
// So it misses where lengths are very uneven in two requests and where few CTAs
// have short contexts: the limit of 1024 keys is for GPUs that are full already.
// It does not look at d, though four CTAs an SM run at d = 64.
int decode_q4_splits(int B, int H, int Hkv, long long max_ctx) {
  const int G = H / Hkv, nh = G <= 8 ? 8 : 16;
  const long long pairs = static_cast<long long>(B) * Hkv * ((G + nh - 1) / nh);
  const long long wave = 152 * (nh == 8 ? 3 : 2);
  long long s = (B <= 2 ? 1 : 3) * wave / pairs;
  const long long most = (max_ctx + 1023) / 1024;
  if (s > most) s = most;
  return s < 1 ? 1 : s > 4096 ? 4096 : static_cast<int>(s);
}

cudaError_t launch_decode_q4(const DecodeQ4& p, int d, int S, cudaStream_t stream) {
  cudaError_t e = d == 64 ? decq4::launch<64>(p, S, stream) : decq4::launch<128>(p, S, stream);
  if (e != cudaSuccess || S == 1) return e;  // one split: the kernel wrote o and lse
  return launch_attn_merge(p.o_part, p.lse_part, S, p.o, p.lse, static_cast<long long>(p.B) * p.H, d, stream);
}

cudaError_t read_and_clear_decode_q4_error(uint32_t* out, cudaStream_t stream) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_decq4_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbolAsync(g_decq4_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return e;
  return cudaStreamSynchronize(stream);
}

}  // namespace fa
