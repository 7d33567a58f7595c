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

#include "fa_common.h"
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

// Makes the compiler take r for new values, so that it does not keep what it
// unpacked from it before.
__device__ __forceinline__ void forget(Raw& r) {
  asm volatile("" : "+r"(r.a.x), "+r"(r.a.y), "+r"(r.a.z), "+r"(r.a.w), "+r"(r.b.x), "+r"(r.b.y), "+r"(r.b.z), "+r"(r.b.w));
}

// Rows are read once and written once: they are kept out of L1.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void store16(void* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// A lane's 16 values as fp32 pairs: one packed instruction works on two.
struct Row {
  float2 a[4], b[4];
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float2 bf_pair(uint32_t v) { return make_float2(bf_lo(v), bf_hi(v)); }

__device__ __forceinline__ void unpack8(const uint4& v, float2* x) {
  x[0] = bf_pair(v.x), x[1] = bf_pair(v.y), x[2] = bf_pair(v.z), x[3] = bf_pair(v.w);
}
__device__ __forceinline__ Row unpack(const Raw& r) {
  Row x;
  unpack8(r.a, x.a);
  unpack8(r.b, x.b);
  return x;
}
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}

// 8 consecutive weights, bf16 or fp32.
__device__ __forceinline__ void load_weight8(const void* w, bool w32, int chunk, float2* out) {
  if (w32) {
    const float4* p = reinterpret_cast<const float4*>(w) + chunk * 2;
    const float4 u = p[0], v = p[1];
    out[0] = make_float2(u.x, u.y), out[1] = make_float2(u.z, u.w);
    out[2] = make_float2(v.x, v.y), out[3] = make_float2(v.z, v.w);
  } else {
    unpack8(reinterpret_cast<const uint4*>(w)[chunk], out);
  }
}

// A lane's 16 fp32 values in shared memory, four by four STRIDE apart, read
// each time.
template <int STRIDE>
__device__ __forceinline__ Row shared_row(const float* p) {
  Row x;
  float2* out[2] = {x.a, x.b};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2* o = out[i >> 1] + 2 * (i & 1);
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(o[0].x), "=f"(o[0].y), "=f"(o[1].x), "=f"(o[1].y)
                 : "r"(smem_u32(p + i * STRIDE)));
  }
  return x;
}

// Sum over the LPR lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Σ x y over a lane's 16 values, in two chains.
__device__ __forceinline__ float dot(const Row& x, const Row& y) {
  float2 u = fmul2(x.a[0], y.a[0]), v = fmul2(x.b[0], y.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    u = ffma2(x.a[i], y.a[i], u);
    v = ffma2(x.b[i], y.b[i], v);
  }
  u = fadd2(u, v);
  return u.x + u.y;
}
__device__ __forceinline__ Row times(const Row& x, const Row& y) {
  Row z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.a[i] = fmul2(x.a[i], y.a[i]), z.b[i] = fmul2(x.b[i], y.b[i]);
  return z;
}
__device__ __forceinline__ Row times(const Row& x, float y) {
  Row z;
  const float2 y2 = make_float2(y, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) z.a[i] = fmul2(x.a[i], y2), z.b[i] = fmul2(x.b[i], y2);
  return z;
}

// 1 / sqrt(mean x² + eps) of a row of 16 LPR values.
template <int LPR>
__device__ __forceinline__ float inv_rms(const Row& x, float eps) {
  return rsqrtf(row_sum<LPR>(dot(x, x)) * (1.f / (16 * LPR)) + eps);
}

// A token's positions on the axes; ok: all of them are rows of the tables.
struct AxisRows {
  int at[4];
  bool ok;
  __device__ __forceinline__ AxisRows(const Axes& x, long long i, int n_pos, uint32_t* err) : ok(true) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      at[a] = 0;
      if (a < x.n) {
        at[a] = in_range(a * x.stride + i, 1, x.n * x.stride, err) ? x.positions[a * x.stride + i] : -1;
        ok = ok && at[a] >= 0 && at[a] < n_pos;
      }
    }
  }
  __device__ __forceinline__ long long row(uint32_t axis) const {
    return axis == 0 ? at[0] : axis == 1 ? at[1] : axis == 2 ? at[2] : at[3];
  }
};

// The cosines and sines a lane needs, from row `pos` of the tables
// ([n_pos][rot/2] fp32). Split: angles 8·ca .. 8·ca + 7 for its eight pairs.
// Interleaved: angles 4·ca .. 4·ca + 3, then 4·cb .. 4·cb + 3.
struct Angles {
  float2 c[4], s[4];
  __device__ __forceinline__ void load(const float* cos, const float* sin, long long pos, int rot, const Lane& ln,
                                       bool interleaved) {
    const long long base = pos * (rot >> 1);
    const int i0 = interleaved ? 4 * ln.ca : 8 * ln.ca;
    const int i1 = interleaved ? 4 * ln.cb : 8 * ln.ca + 4;
    const float4 c0 = *reinterpret_cast<const float4*>(cos + base + i0);
    const float4 c1 = *reinterpret_cast<const float4*>(cos + base + i1);
    const float4 s0 = *reinterpret_cast<const float4*>(sin + base + i0);
    const float4 s1 = *reinterpret_cast<const float4*>(sin + base + i1);
    c[0] = make_float2(c0.x, c0.y), c[1] = make_float2(c0.z, c0.w);
    c[2] = make_float2(c1.x, c1.y), c[3] = make_float2(c1.z, c1.w);
    s[0] = make_float2(s0.x, s0.y), s[1] = make_float2(s0.z, s0.w);
    s[2] = make_float2(s1.x, s1.y), s[3] = make_float2(s1.z, s1.w);
  }
  // The same with each pair's row of its own axis: four at once where four
  // neighbours share one (sections of multiples of 4), else one by one.
  __device__ __forceinline__ void load(const float* cos, const float* sin, const AxisRows& rows, const Axes& axes,
                                       int rot, const Lane& ln, bool interleaved) {
    const int half = rot >> 1;
    const int first[2] = {interleaved ? 4 * ln.ca : 8 * ln.ca, interleaved ? 4 * ln.cb : 8 * ln.ca + 4};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = first[q];
      const uint32_t bits = static_cast<uint32_t>((i < 32 ? axes.of_pair[0] : axes.of_pair[1]) >> (2 * (i & 31))) & 0xffu;
      float4 c4, s4;
      if (bits == (bits & 3u) * 0x55u) {
        const long long base = rows.row(bits & 3u) * half + i;
        c4 = *reinterpret_cast<const float4*>(cos + base);
        s4 = *reinterpret_cast<const float4*>(sin + base);
      } else {
        const long long b0 = rows.row(bits & 3u) * half + i, b1 = rows.row(bits >> 2 & 3u) * half + i + 1;
        const long long b2 = rows.row(bits >> 4 & 3u) * half + i + 2, b3 = rows.row(bits >> 6) * half + i + 3;
        c4 = make_float4(cos[b0], cos[b1], cos[b2], cos[b3]);
        s4 = make_float4(sin[b0], sin[b1], sin[b2], sin[b3]);
      }
      c[2 * q] = make_float2(c4.x, c4.y), c[2 * q + 1] = make_float2(c4.z, c4.w);
      s[2 * q] = make_float2(s4.x, s4.y), s[2 * q + 1] = make_float2(s4.z, s4.w);
    }
  }
};

// (a, b) -> (a c − b s, b c + a s) for the pair in one float2. Each product
// and sum of a rotation is rounded by itself, never contracted: a key's
// values, and with them the codes of a 4-bit cache, then do not hang on how a
// compiler fuses the expression, and every kernel here gives the same bits.
// (Packed sums of packed products are contracted, whatever their rounding
// says: one key group's step in 10^4 came out a bf16 step off. So products
// are packed, sums are not.)
__device__ __forceinline__ float2 turn1(float2 x, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s)), __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s)));
}

// Turn a lane's values; BACK turns back.
template <bool BACK>
__device__ __forceinline__ void turn(Row& x, const Angles& t, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 s = BACK ? make_float2(-t.s[i].x, -t.s[i].y) : t.s[i];
    if (interleaved) {
      float2* half = i < 2 ? x.a : x.b;  // pairs 2i and 2i + 1 of the lane
      half[2 * (i & 1)] = turn1(half[2 * (i & 1)], t.c[i].x, s.x);
      half[2 * (i & 1) + 1] = turn1(half[2 * (i & 1) + 1], t.c[i].y, s.y);
    } else {
      const float2 ac = fmul2(x.a[i], t.c[i]), bs = fmul2(x.b[i], s), bc = fmul2(x.b[i], t.c[i]), as = fmul2(x.a[i], s);
      x.a[i] = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
      x.b[i] = make_float2(__fadd_rn(bc.x, as.x), __fadd_rn(bc.y, as.y));
    }
  }
}

}  // namespace rope
}  // namespace fa
