// 4-bit codes of cached keys and values. A row of D values is cut into
// groups of 64; each group has a step s and a centre z (bf16 both) and a
// code n in 0..15 per value, standing for z + s (n − 8). For the group's
// smallest and largest values a and b:
//     s = bf16((b − a)/2 · (1/7.5)),  z = bf16((a + b)/2 + s/2),
//     n = clamp(rint((x − z) / s) + 8, 0, 15)       (n = 8 where s = 0)
// so the 16 levels span a .. b up to the rounding of s and z, and a value is
// off by at most max(s/2, 2^-8 (|z| + 8 s)) (the second where the rounding
// of z or s shifts the end levels by more than half a step). s and z are
// bf16 because the values are: their range is bf16's (fp16 would overflow),
// and the levels are then no coarser than bf16 values of that size. A group
// with a value that is not finite has s = z = NaN, n = 8. The centre is kept,
// not the smallest value: attention sums over s (n − 8), whose rounding
// errors then go with the spread of a group, not with its offset.
//
// Codes are packed two a byte, the even dimension in the low half, so 8
// consecutive dimensions are one 32-bit word; the pair (s, z) is one too.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "fa_rope.cuh"

namespace fa {
namespace q4 {

constexpr int GROUP = 64;

struct Grid {
  float s, z;
};

// Smallest and largest of two or three, NaN if any is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float round_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// Step and centre of a group with smallest value a and largest b. Each
// operation is rounded by itself (no contraction), so the codes are a
// function of the values alone.
__device__ __forceinline__ Grid grid_of(float a, float b) {
  const float half = __fsub_rn(0.5f * b, 0.5f * a);  // halves first: b − a may overflow
  Grid g;
  g.s = round_bf16(__fmul_rn(half, 1.f / 7.5f));
  g.z = round_bf16(__fadd_rn(__fadd_rn(0.5f * a, 0.5f * b), 0.5f * g.s));
  if (!(half < INFINITY) || !(fabsf(g.z) < INFINITY)) g.s = g.z = __int_as_float(0x7fffffff);
  return g;
}

__device__ __forceinline__ uint32_t pair(const Grid& g) { return pack_bf16x2(g.s, g.z); }

// The group that lane i of a row works out (and writes the pair of).
template <int D>
__device__ __forceinline__ int own_group(int i) {
  return D == GROUP ? 0 : i / (D / 32);
}

// The groups' grids of a row whose lanes hold chunks ln.ca and ln.cb; every
// lane of the row gets all of them. With two groups each half of the lanes
// reduces one (the first exchange hands over the other's part) and the halves
// swap the results.
template <int D>
__device__ __forceinline__ void grids(const rope::Row& x, const rope::Lane& ln, int i, Grid (&out)[D / GROUP]) {
  constexpr int LPR = D / 16, NG = D / GROUP;
  float la = x.a[0].x, ha = la, lb = x.b[0].x, hb = lb;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    la = min_nan3(la, x.a[e].x, x.a[e].y), ha = max_nan3(ha, x.a[e].x, x.a[e].y);
    lb = min_nan3(lb, x.b[e].x, x.b[e].y), hb = max_nan3(hb, x.b[e].x, x.b[e].y);
  }
  const unsigned all = 0xffffffffu;
  float lo, hi;
  if constexpr (NG == 1) {
    lo = min_nan(la, lb), hi = max_nan(ha, hb);
  } else {
    const int mine = own_group<D>(i);
    float l[2] = {INFINITY, INFINITY}, h[2] = {-INFINITY, -INFINITY};  // [kept, handed over]
    const bool a_mine = ln.ca / 8 == mine, b_mine = ln.cb / 8 == mine;
    l[0] = min_nan(a_mine ? la : INFINITY, b_mine ? lb : INFINITY);
    h[0] = max_nan(a_mine ? ha : -INFINITY, b_mine ? hb : -INFINITY);
    l[1] = min_nan(a_mine ? INFINITY : la, b_mine ? INFINITY : lb);
    h[1] = max_nan(a_mine ? -INFINITY : ha, b_mine ? -INFINITY : hb);
    lo = min_nan(l[0], __shfl_xor_sync(all, l[1], LPR / 2));
    hi = max_nan(h[0], __shfl_xor_sync(all, h[1], LPR / 2));
  }
#pragma unroll
  for (int o = NG == 1 ? LPR / 2 : LPR / 4; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(all, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(all, hi, o));
  }
  const Grid own = grid_of(lo, hi);
  if constexpr (NG == 1) {
    out[0] = own;
  } else {
    const uint32_t other = __shfl_xor_sync(all, pair(own), LPR / 2);
    const Grid g{rope::bf_lo(other), rope::bf_hi(other)};
    const bool first = own_group<D>(i) == 0;
    out[0] = first ? own : g;
    out[1] = first ? g : own;
  }
}

// Eight codes as one word; n gets the levels n − 8. The level is the quotient
// (x − z) / s rounded to fp32, then to a whole number: bf16 values often lie
// exactly between two levels, and a product with 1/s would send them either
// way. The quotient comes from the product and one correction by its residual
// (Markstein, 1990): with y = 1/s rounded and q = d y, d − q s is exact and
// q + (d − q s) y is off the true quotient by 2^-22 of a last place before its
// rounding. s has 8 significant bits, so d / s is never halfway between two
// fp32 values and never nearer to it than 2^-9 of a last place: the rounded
// sum is the rounded quotient. Far from the normal range's ends, that is:
// below s = 2^-60 it is divided. (16384 prompt tokens: 108 us with divisions,
// 88 so.)
__device__ __forceinline__ uint32_t encode8(const float2* x, const Grid& g, float2* n) {
  if (!(g.s > 0.f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = make_float2(0.f, 0.f);
    return 0x88888888u;
  }
  constexpr float ROUND = 12582912.f;  // 1.5 · 2^23: adding it rounds to a whole number, in the low bits
  const float2 z2 = make_float2(g.z, g.z), s2 = make_float2(-g.s, -g.s), round2 = make_float2(ROUND, ROUND);
  if (g.s >= 0x1p-60f) {
    const float y = __frcp_rn(g.s);
    const float2 y2 = make_float2(y, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (A normed key's product with its weight reaches here through the
      // rotation's branch, so it is rounded before this difference.)
      const float2 d = fsub2(x[e], z2), q = fmul2(d, y2);
      n[e] = ffma2(ffma2(q, s2, d), y2, q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      n[e] = make_float2(__fdiv_rn(__fsub_rn(x[e].x, g.z), g.s), __fdiv_rn(__fsub_rn(x[e].y, g.z), g.s));
  }
  // 16^e-weighted sum of the codes, each with ROUND's bits above it, which
  // add up to a constant.
  uint32_t w = 0;
#pragma unroll
  for (int e = 3; e >= 0; --e) {
    n[e] = make_float2(fminf(fmaxf(n[e].x, -8.f), 7.f), fminf(fmaxf(n[e].y, -8.f), 7.f));
    const float2 whole = fadd2(n[e], round2);
    n[e] = fsub2(whole, round2);
    w = w * 16u + __float_as_uint(whole.y);
    w = w * 16u + __float_as_uint(whole.x);
  }
  return w - 0xb6b77778u;
}

// The values held: z + s n, rounded once to fp32.
__device__ __forceinline__ void held8(const float2* n, const Grid& g, float2* x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = ffma2(n[e], make_float2(g.s, g.s), make_float2(g.z, g.z));
}

}  // namespace q4
}  // namespace fa
