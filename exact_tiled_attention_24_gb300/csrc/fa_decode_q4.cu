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
// The step is bound by reading the codes: d/2 + d/16 bytes a key or value.
// At 6.8 TB/s an SM takes in 23 bytes a clock, 47 values, and each has to be
// turned into an operand. tcgen05 takes operands from shared memory or TMEM,
// and writing 47 bf16 values a clock there and reading them back is more than
// shared memory's 128 bytes a clock. So a warp keeps them in registers:
// mma.sync m16n8k16, whose A operand is 16 keys (scores) or 16 dimensions
// (output) and whose 8 columns are query heads that share the K/V head.
//   scores  Sᵀ[key][head]: rows g and g + 8 of a tile are keys; the words of
//           a key's row go to the lane quarter t that needs them as they are
//           (the order of the products' inner index is free: q is read in
//           the same order).
//   output  Oᵀ[dim][head]: an operand register pairs two keys of one
//           dimension, two words' halves merged by one byte permutation.
// A nibble becomes a bf16 number by placing it in the top four mantissa bits
// of 16.0 (16 + n: one shift, one and-or for two values). The scores keep
// that offset and take it off with the centre (s Σ q (16 + n) + (z − 24 s) Σ q);
// the values subtract it first, since their sums run over the whole context.
// Each warp walks its own 16-key tiles; the CTA's warps are merged at its end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_ptx.cuh"

namespace fa {

static __device__ uint32_t g_decq4_err;

namespace decq4 {

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int TK = 16;  // keys per warp tile
constexpr float LN2 = 0.69314718055994531f;
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t NO_ROW = 0xffffffffu;

// d (+)= A (16x16 bf16) B (16x8 bf16), fp32.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// 16 + n for nibble I of each 16-bit half, as two bf16.
template <int I>
__device__ __forceinline__ uint32_t nibbles16(uint32_t w) {
  const uint32_t v = I == 0 ? w << 3 : w >> (4 * I - 3);
  return (v & 0x00780078u) | 0x41804180u;
}
// n − 8 (exact: both are bf16 integers).
template <int I>
__device__ __forceinline__ uint32_t nibbles_centred(uint32_t w) {
  uint32_t v = nibbles16<I>(w), d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x41c041c0u));  // 24
  return d;
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// One CTA: split s of request b's context, K/V head hk, 8·NT query heads.
template <int D, int NT>
__global__ void __launch_bounds__(THREADS) decode_q4_kernel(const DecodeQ4 p) {
  constexpr int NG = D / 64;    // groups of a row
  constexpr int NH = 8 * NT;    // query heads of the CTA
  constexpr int MT = D / 16;    // 16-dimension tiles of the output
  __shared__ float sm_o[WARPS][NH][D + 1];
  __shared__ float sm_m[WARPS][NH], sm_l[WARPS][NH];
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
  const int n_tiles = (L + TK - 1) / TK;
  const int tps = (n_tiles + S - 1) / S;
  const int tile0 = s * tps, tile1 = min(n_tiles, tile0 + tps);

  // Query operand: for group gr and word w of a lane quarter's 16 dimensions
  // 64 gr + 16 t + 8 w + 0..7, K step 2 h' (h' = 0, 1) multiplies elements
  // (2h', 2h'+4) and (2h'+1, 2h'+5).
  uint32_t qf[NT][NG][4][2];
  float qsum[NT][NG][2];  // Σ q over a group, of this lane's heads 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const long long off = static_cast<long long>(head0 + nt * 8 + g) * D + gr * 64 + t * 16 + w * 8;
        if (nt * 8 + g < G && in_range(off, 8, static_cast<long long>(p.B) * p.H * D, err))
          v = *reinterpret_cast<const uint4*>(p.q + off);
        // v.x = (e0, e1), v.y = (e2, e3), v.z = (e4, e5), v.w = (e6, e7)
        qf[nt][gr][2 * w][0] = __byte_perm(v.x, v.z, 0x5410);
        qf[nt][gr][2 * w][1] = __byte_perm(v.x, v.z, 0x7632);
        qf[nt][gr][2 * w + 1][0] = __byte_perm(v.y, v.w, 0x5410);
        qf[nt][gr][2 * w + 1][1] = __byte_perm(v.y, v.w, 0x7632);
      }
      const uint32_t one = 0x3f803f80u;
      const uint32_t ones[4] = {one, one, one, one};
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma(c, ones, qf[nt][gr][ks][0], qf[nt][gr][ks][1]);
      qsum[nt][gr][0] = c[0];
      qsum[nt][gr][1] = c[1];
    }

  float acc[NT][MT][4];
  float m[NT][2], l[NT][2], zc[NT][NG][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) zc[nt][gr][e] = 0.f;
    }
  }

  const long long rows = static_cast<long long>(p.num_blocks) * p.Hkv * p.bs;
  for (int tile = tile0 + warp; tile < tile1; tile += WARPS) {
    // Lanes 0..15 look up the tile's rows of the cache.
    uint32_t row = NO_ROW;
    {
      const int tok = tile * TK + (lane & 15);
      if (tok < L) {
        const int bi = tok / p.bs;
        const long long ti = static_cast<long long>(b) * p.max_blocks + bi;
        const int blk = in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err) ? p.block_table[ti] : -1;
        if (blk >= 0 && blk < p.num_blocks)
          row = (static_cast<uint32_t>(blk) * p.Hkv + hk) * static_cast<uint32_t>(p.bs) +
                static_cast<uint32_t>(tok - bi * p.bs);
        else
          atomicExch(err, DEV_BAD_INDEX);
      }
    }
    uint32_t krow[2], vrow[4];
    krow[0] = __shfl_sync(0xffffffffu, row, g);
    krow[1] = __shfl_sync(0xffffffffu, row, g + 8);
    vrow[0] = __shfl_sync(0xffffffffu, row, 2 * t);
    vrow[1] = __shfl_sync(0xffffffffu, row, 2 * t + 1);
    vrow[2] = __shfl_sync(0xffffffffu, row, 2 * t + 8);
    vrow[3] = __shfl_sync(0xffffffffu, row, 2 * t + 9);

    uint2 kw[2][NG];
    uint32_t ks_[2][NG], vs_[2][NG], vw[4][NG];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        kw[r][gr] = make_uint2(0, 0);
        ks_[r][gr] = vs_[r][gr] = 0;
        if (krow[r] != NO_ROW) {
          const long long c = static_cast<long long>(krow[r]) * (D / 2) + gr * 32 + t * 8;
          const long long sc = static_cast<long long>(krow[r]) * NG + gr;
          if (in_range(c, 8, rows * (D / 2), err)) kw[r][gr] = *reinterpret_cast<const uint2*>(p.k_cache + c);
          if (in_range(sc, 1, rows * NG, err)) {
            ks_[r][gr] = p.k_scale[sc];
            vs_[r][gr] = p.v_scale[sc];
          }
        }
      }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        vw[r][gr] = 0;
        const long long c = static_cast<long long>(vrow[r]) * (D / 2) + gr * 32 + g * 4;
        if (vrow[r] != NO_ROW && in_range(c, 4, rows * (D / 2), err))
          vw[r][gr] = *reinterpret_cast<const uint32_t*>(p.v_cache + c);
      }

    // Scores, in log2 units: x[nt][2 r + e] is key g + 8 r, head 2 t + e.
    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t a[4][4];  // per K step
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        a[0][r] = nibbles16<0>(kw[r][gr].x), a[0][r + 2] = nibbles16<1>(kw[r][gr].x);
        a[1][r] = nibbles16<2>(kw[r][gr].x), a[1][r + 2] = nibbles16<3>(kw[r][gr].x);
        a[2][r] = nibbles16<0>(kw[r][gr].y), a[2][r + 2] = nibbles16<1>(kw[r][gr].y);
        a[3][r] = nibbles16<2>(kw[r][gr].y), a[3][r + 2] = nibbles16<3>(kw[r][gr].y);
      }
      float st[2], zt[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st[r] = bf_lo(ks_[r][gr]) * p.scale_log2;
        zt[r] = fmaf(-24.f, st[r], bf_hi(ks_[r][gr]) * p.scale_log2);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma(c, a[ks], qf[nt][gr][ks][0], qf[nt][gr][ks][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[nt][e] += fmaf(st[e >> 1], c[e], zt[e >> 1] * qsum[nt][gr][e & 1]);
      }
    }
    bool need = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (krow[e >> 1] == NO_ROW) x[nt][e] = -INFINITY;
        need |= x[nt][e] > m[nt][e & 1] + RESCALE_LOG2;
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(x[nt][e], x[nt][e + 2]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          const float m_new = fmaxf(m[nt][e], v);
          const float alpha = m_new == -INFINITY ? 1.f : ex2(m[nt][e] - m_new);
          m[nt][e] = m_new;
          l[nt][e] *= alpha;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) zc[nt][gr][e] *= alpha;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[nt][i][e] *= alpha;
            acc[nt][i][e + 2] *= alpha;
          }
        }
    }
    // Probabilities, times the values' steps, as the output's B operand.
    uint32_t pf[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pr[e] = krow[e >> 1] == NO_ROW ? 0.f : ex2(x[nt][e] - m[nt][e & 1]);
        l[nt][e & 1] += pr[e];
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sv = bf_lo(vs_[r][gr]), zv = bf_hi(vs_[r][gr]);
          zc[nt][gr][0] = fmaf(pr[2 * r], zv, zc[nt][gr][0]);
          zc[nt][gr][1] = fmaf(pr[2 * r + 1], zv, zc[nt][gr][1]);
          // bf16: its range takes any step, and the products' errors
          // (2^-9 each) average out over the keys.
          pf[nt][gr][r] = transpose8x8(pack_bf16x2(pr[2 * r] * sv, pr[2 * r + 1] * sv));
        }
    }
    // Output: tile 4 gr + i has dimension 64 gr + 8 g + i in row g, + 4 in row g + 8.
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const uint32_t lo0 = __byte_perm(vw[0][gr], vw[1][gr], 0x5410), hi0 = __byte_perm(vw[0][gr], vw[1][gr], 0x7632);
      const uint32_t lo1 = __byte_perm(vw[2][gr], vw[3][gr], 0x5410), hi1 = __byte_perm(vw[2][gr], vw[3][gr], 0x7632);
      const uint32_t a0[4] = {nibbles_centred<0>(lo0), nibbles_centred<0>(hi0), nibbles_centred<0>(lo1), nibbles_centred<0>(hi1)};
      const uint32_t a1[4] = {nibbles_centred<1>(lo0), nibbles_centred<1>(hi0), nibbles_centred<1>(lo1), nibbles_centred<1>(hi1)};
      const uint32_t a2[4] = {nibbles_centred<2>(lo0), nibbles_centred<2>(hi0), nibbles_centred<2>(lo1), nibbles_centred<2>(hi1)};
      const uint32_t a3[4] = {nibbles_centred<3>(lo0), nibbles_centred<3>(hi0), nibbles_centred<3>(lo1), nibbles_centred<3>(hi1)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(acc[nt][4 * gr], a0, pf[nt][gr][0], pf[nt][gr][1]);
        mma(acc[nt][4 * gr + 1], a1, pf[nt][gr][0], pf[nt][gr][1]);
        mma(acc[nt][4 * gr + 2], a2, pf[nt][gr][0], pf[nt][gr][1]);
        mma(acc[nt][4 * gr + 3], a3, pf[nt][gr][0], pf[nt][gr][1]);
      }
    }
  }

  // The warps' results: Σ over the lanes that hold other keys, then one
  // (m, l, o) per head and warp in shared memory.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = nt * 8 + 2 * t + e;
      float lv = l[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lv += __shfl_xor_sync(0xffffffffu, lv, o);
      if (g == 0) {
        sm_m[warp][h] = m[nt][e];
        sm_l[warp][h] = lv;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float z = zc[nt][gr][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sm_o[warp][h][64 * gr + 8 * g + i] = acc[nt][4 * gr + i][e] + z;
          sm_o[warp][h][64 * gr + 8 * g + i + 4] = acc[nt][4 * gr + i][e + 2] + z;
        }
      }
    }
  __syncthreads();
  for (int idx = threadIdx.x; idx < G * D; idx += THREADS) {
    const int h = idx / D, c = idx % D;
    float mm = sm_m[0][h];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mm = fmaxf(mm, sm_m[w][h]);
    float lt = 0.f, ot = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      // l = 0: a warp that saw no key (and o = 0). A NaN score leaves l NaN,
      // whatever m is, and the head's result with it.
      const float a = sm_l[w][h] == 0.f ? 0.f : ex2(sm_m[w][h] - mm);
      lt = fmaf(a, sm_l[w][h], lt);
      ot = fmaf(a, sm_o[w][h][c], ot);
    }
    const bool any = lt != 0.f;
    const float ov = any ? ot / lt : 0.f;
    const long long orow = prow + h;
    if (in_range(orow * D + c, 1, part_rows * D, err)) {
      if (S == 1) p.o[orow * D + c] = __float2bfloat16_rn(ov);
      else p.o_part[orow * D + c] = ov;
    }
    if (c == 0 && in_range(orow, 1, part_rows, err))
      (S == 1 ? p.lse : p.lse_part)[orow] = any ? (mm + __log2f(lt)) * LN2 : -INFINITY;
  }
}

template <int D>
static cudaError_t launch(const DecodeQ4& p, int S, cudaStream_t stream) {
  const int G = p.H / p.Hkv;
  const int nt = G <= 8 ? 1 : 2, n_chunk = (G + 8 * nt - 1) / (8 * nt);
  const dim3 grid(static_cast<unsigned>(S), static_cast<unsigned>(p.Hkv * n_chunk), static_cast<unsigned>(p.B));
  if (nt == 1) decode_q4_kernel<D, 1><<<grid, THREADS, 0, stream>>>(p);
  else decode_q4_kernel<D, 2><<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace decq4

int decode_q4_splits(int B, int H, int Hkv, long long max_ctx) {
  const int G = H / Hkv, nh = G <= 8 ? 8 : 16;
  const long long ctas = static_cast<long long>(B) * Hkv * ((G + nh - 1) / nh);
  long long s = (152 * 8 + ctas - 1) / ctas;                       // about eight CTAs per SM
  const long long most = (max_ctx + 255) / 256;                    // at least 256 keys a split
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
