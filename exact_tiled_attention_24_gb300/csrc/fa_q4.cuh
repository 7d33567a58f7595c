// 4-bit codes of cached keys and values. A row of D values is cut into
// groups of 64; each group has a step s and a centre z (bf16 both) and a
// code n in 0..15 per value, standing for z + s (n − 8). For the group's
// smallest and largest values a and b:
//     s = bf16((b − a)/2 · (1/7.5)),  z = bf16((a + b)/2 + s/2),
//     n = clamp(rint((x − z) / s) + 8, 0, 15)       (n = 8 where s = 0)
// so the 16 levels span a .. b up to the rounding of s and z, and a value is
// off by at most max(s/2, 2^-9 (|z| + 8 s)) (the second where the rounding
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

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if either is
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
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

// The groups' grids of a row whose lanes hold chunks a (ln.ca) and b
// (ln.cb): every lane of the row gets all of them.
template <int D>
__device__ __forceinline__ void grids(const float* a, const float* b, const rope::Lane& ln, Grid* out) {
  constexpr int LPR = D / 16, NG = D / GROUP;
  float la = a[0], ha = a[0], lb = b[0], hb = b[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    la = min_nan(la, a[e]), ha = max_nan(ha, a[e]);
    lb = min_nan(lb, b[e]), hb = max_nan(hb, b[e]);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float lo = INFINITY, hi = -INFINITY;
    if (NG == 1 || ln.ca / 8 == g) lo = min_nan(lo, la), hi = max_nan(hi, ha);
    if (NG == 1 || ln.cb / 8 == g) lo = min_nan(lo, lb), hi = max_nan(hi, hb);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    out[g] = grid_of(lo, hi);
  }
}

// Eight codes as one word. A division, not a product with 1/s: bf16 values
// often lie exactly between two levels, and the reciprocal's rounding would
// send them either way.
__device__ __forceinline__ uint32_t encode8(const float* x, const Grid& g) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int n = 8;
    if (g.s > 0.f) n = min(max(__float2int_rn(__fdiv_rn(__fsub_rn(x[e], g.z), g.s)) + 8, 0), 15);
    w |= static_cast<uint32_t>(n) << (4 * e);
  }
  return w;
}

// The values held: z + s (n − 8), rounded once to fp32.
__device__ __forceinline__ void decode8(uint32_t w, const Grid& g, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    x[e] = fmaf(g.s, static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8), g.z);
}

__device__ __forceinline__ uint32_t pair(const Grid& g) { return pack_bf16x2(g.s, g.z); }

}  // namespace q4
}  // namespace fa
