// One row (one head of one token) of the norm and rotation kernels.
//
//   norm      r = 1 / sqrt(mean_c x_c² + eps),  y_c = x_c · r · w_c
//   rotation  pairs (a, b) of y turn by the token's angle of that pair:
//             (a, b) -> (a cos − b sin, b cos + a sin).  With rot rotated
//             dimensions, pair i is (i, i + rot/2), or (2i, 2i + 1) in the
//             interleaved form; dimensions from rot on pass through.
//
// D / 16 lanes share a row and each holds two chunks of 8 elements (16
// bytes in bf16), chosen so that both members of a split pair sit in one
// lane: no exchange between lanes but the row sums. Everything is fp32 from
// the loads to the one rounding of the result.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "fa_ptx.cuh"

namespace fa {
namespace rope {

// The two chunks lane i of a row holds, for rot rotated dimensions: chunks
// i and i + rot/16 (the two halves of eight split pairs), then the chunks
// that pass through two by two. rot = 0: chunks 2i and 2i + 1.
struct Lane {
  int ca, cb;    // chunk indices
  bool turned;   // the chunks are rotated
  __device__ __forceinline__ Lane(int i, int rot) {
    const int half = rot >> 4;
    turned = i < half;
    ca = turned ? i : 2 * i;  // the first 2·half chunks are the turned ones
    cb = turned ? i + half : ca + 1;
  }
};

struct Raw {  // the two chunks as loaded
  uint4 a, b;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
  x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 8 consecutive weights, bf16 or fp32.
__device__ __forceinline__ void load_weight8(const void* w, bool w32, int chunk, float* out) {
  if (w32) {
    const float4* p = reinterpret_cast<const float4*>(w) + chunk * 2;
    const float4 u = p[0], v = p[1];
    out[0] = u.x, out[1] = u.y, out[2] = u.z, out[3] = u.w;
    out[4] = v.x, out[5] = v.y, out[6] = v.z, out[7] = v.w;
  } else {
    unpack8(reinterpret_cast<const uint4*>(w)[chunk], out);
  }
}

// Sum over the LPR lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The cosines and sines a lane needs, from row `pos` of the tables
// ([n_pos][rot/2] fp32). Split: angles 8·ca .. 8·ca + 7 for its eight pairs.
// Interleaved: angles 4·ca .. 4·ca + 3, then 4·cb .. 4·cb + 3.
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* cos, const float* sin, long long pos, int rot, const Lane& ln,
                                       bool interleaved) {
    const long long base = pos * (rot >> 1);
    const int i0 = interleaved ? 4 * ln.ca : 8 * ln.ca;
    const int i1 = interleaved ? 4 * ln.cb : 8 * ln.ca + 4;
    const float4 c0 = *reinterpret_cast<const float4*>(cos + base + i0);
    const float4 c1 = *reinterpret_cast<const float4*>(cos + base + i1);
    const float4 s0 = *reinterpret_cast<const float4*>(sin + base + i0);
    const float4 s1 = *reinterpret_cast<const float4*>(sin + base + i1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
};

// (a, b) -> (a c − b s, b c + a s). Each product and sum is rounded by
// itself, never contracted: a key's values, and with them the codes of a
// 4-bit cache, then do not hang on how a compiler fuses the expression.
__device__ __forceinline__ void turn1(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

// Turn the lane's chunks a (ca) and b (cb); sign = -1 turns back.
__device__ __forceinline__ void turn(float* a, float* b, const Angles& t, bool interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn1(a[2 * i], a[2 * i + 1], t.c[i], sign * t.s[i]);
      turn1(b[2 * i], b[2 * i + 1], t.c[4 + i], sign * t.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn1(a[i], b[i], t.c[i], sign * t.s[i]);
  }
}

}  // namespace rope
}  // namespace fa
