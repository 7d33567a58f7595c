// Per-head norms of q and k with the position rotation in the same pass, and
// their gradient: what stands between a layer's projections and the
// attention forward (fa_rope.cuh has the formulas of one row).
//
// Gradient of one row for the output gradient dy, with g = Rᵀ dy (the
// rotation turned back), n = x r (the normed row) and h = g w:
//     dx = r (h − n · mean_c(h_c n_c)),     dw = Σ_rows g n.
// x is read again and r formed again from it: saving r would cost a write
// and a read of 4 bytes per row against nothing but a sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_rope.cuh"

namespace fa {

static __device__ uint32_t g_rope_err;

namespace rope {

constexpr int THREADS = 256;

// Row of a strided [B][heads][N][D] tensor as two 16-byte chunks.
__device__ __forceinline__ Raw load_row(const HeadRows& t, long long off, const Lane& ln, uint32_t* err) {
  Raw r{};
  if (in_range(off + ln.ca * 8, 8, t.extent, err)) r.a = *reinterpret_cast<const uint4*>(t.p + off + ln.ca * 8);
  if (in_range(off + ln.cb * 8, 8, t.extent, err)) r.b = *reinterpret_cast<const uint4*>(t.p + off + ln.cb * 8);
  return r;
}
__device__ __forceinline__ void store_row(const HeadRows& t, long long off, const Lane& ln, const float* a,
                                          const float* b, uint32_t* err) {
  if (in_range(off + ln.ca * 8, 8, t.extent, err)) *reinterpret_cast<uint4*>(t.p + off + ln.ca * 8) = pack8(a);
  if (in_range(off + ln.cb * 8, 8, t.extent, err)) *reinterpret_cast<uint4*>(t.p + off + ln.cb * 8) = pack8(b);
}

// The row of the tables for token (b, n), or -1 (reported) for a position
// outside them.
__device__ __forceinline__ int position_of(const NormRope& p, int b, int n, uint32_t* err) {
  if (p.rot == 0) return 0;
  int pos = n;
  if (p.positions) {
    const long long i = b * p.pos_sb + n;
    pos = in_range(i, 1, p.pos_sb * (p.B - 1) + p.N, err) ? p.positions[i] : -1;
  }
  if (pos >= 0 && pos < p.n_pos) return pos;
  atomicExch(err, DEV_BAD_INDEX);
  return -1;
}

// Forward. A row of lanes takes one token and HPG consecutive heads of q or
// of k (blockIdx.y says which), so the token's angles are read once for
// them; the rows of a warp are consecutive tokens, contiguous in the output.
template <int D, int HPG>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const NormRope p) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR;
  uint32_t* err = &g_rope_err;
  const int i = threadIdx.x % LPR;
  const long long tok = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / LPR;
  const bool live = tok < static_cast<long long>(p.B) * p.N;
  const int b = live ? static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(p.N)) : 0;
  const int n = live ? static_cast<int>(tok - static_cast<long long>(b) * p.N) : 0;
  const bool is_k = static_cast<int>(blockIdx.y) >= p.q_groups;
  const int h0 = (static_cast<int>(blockIdx.y) - (is_k ? p.q_groups : 0)) * HPG;
  const int heads = min(HPG, (is_k ? p.Hkv : p.H) - h0);
  const HeadRows& src = is_k ? p.k : p.q;
  const HeadRows& dst = is_k ? p.k_out : p.q_out;
  const Lane ln(i, p.rot);

  Raw raw[HPG];
#pragma unroll
  for (int j = 0; j < HPG; ++j)
    raw[j] = live && j < heads ? load_row(src, b * src.sb + (h0 + j) * src.sh + n * src.sn, ln, err) : Raw{};
  const int pos = live ? position_of(p, b, n, err) : 0;
  Angles t;
  if (ln.turned && pos >= 0) t.load(p.cos, p.sin, pos, p.rot, ln, p.interleaved);
  float wa[8], wb[8];
  const void* w = is_k ? p.k_weight : p.q_weight;
  if (w) {
    load_weight8(w, p.w32, ln.ca, wa);
    load_weight8(w, p.w32, ln.cb, wb);
  }
#pragma unroll
  for (int j = 0; j < HPG; ++j) {
    float a[8], c[8];
    unpack8(raw[j].a, a);
    unpack8(raw[j].b, c);
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(c[e], c[e], ss));
      const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * r * wa[e];
        c[e] = c[e] * r * wb[e];
      }
    }
    if (ln.turned && pos >= 0) turn(a, c, t, p.interleaved, 1.f);
    if (pos < 0) {  // no angle to turn by: a zero row
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = c[e] = 0.f;
    }
    if (live && j < heads) store_row(dst, b * dst.sb + (h0 + j) * dst.sh + n * dst.sn, ln, a, c, err);
  }
}

// Backward. blockIdx.y: 0 for q, 1 for k. A CTA walks over (token, head)
// rows of its tensor with its lanes' 16 dimensions of dw in registers, then
// sums them over its rows in a fixed order into one partial row per CTA.
template <int D, bool NORM>
__global__ void __launch_bounds__(THREADS) norm_rope_bwd_kernel(const NormRope p, float* __restrict__ partial) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR, WARPS = THREADS / 32;
  uint32_t* err = &g_rope_err;
  __shared__ float red[WARPS][D];
  const int i = threadIdx.x % LPR;
  const bool is_k = blockIdx.y != 0;
  const HeadRows& x_t = is_k ? p.k : p.q;
  const HeadRows& dy_t = is_k ? p.k_out : p.q_out;
  const HeadRows& dx_t = is_k ? p.dk : p.dq;
  const int heads = is_k ? p.Hkv : p.H;
  const Lane ln(i, p.rot);
  float wa[8], wb[8], dwa[8], dwb[8];
  if (NORM) {
    load_weight8(is_k ? p.k_weight : p.q_weight, p.w32, ln.ca, wa);
    load_weight8(is_k ? p.k_weight : p.q_weight, p.w32, ln.cb, wb);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) dwa[e] = dwb[e] = 0.f;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  for (long long t0 = static_cast<long long>(blockIdx.x) * ROWS; t0 < tokens;
       t0 += static_cast<long long>(gridDim.x) * ROWS) {
    const long long tok = t0 + threadIdx.x / LPR;
    const bool live = tok < tokens;
    const int b = live ? static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(p.N)) : 0;
    const int n = live ? static_cast<int>(tok - static_cast<long long>(b) * p.N) : 0;
    const int pos = live ? position_of(p, b, n, err) : 0;
    Angles t;
    if (ln.turned && pos >= 0) t.load(p.cos, p.sin, pos, p.rot, ln, p.interleaved);
    for (int h = 0; h < heads; ++h) {
      Raw dy{}, x{};
      if (live) {
        dy = load_row(dy_t, b * dy_t.sb + h * dy_t.sh + n * dy_t.sn, ln, err);
        if (NORM) x = load_row(x_t, b * x_t.sb + h * x_t.sh + n * x_t.sn, ln, err);
      }
      float ga[8], gb[8];
      unpack8(dy.a, ga);
      unpack8(dy.b, gb);
      if (ln.turned && pos >= 0) turn(ga, gb, t, p.interleaved, -1.f);
      if (pos < 0) {  // the forward wrote a zero row: no gradient
#pragma unroll
        for (int e = 0; e < 8; ++e) ga[e] = gb[e] = 0.f;
      }
      if (NORM) {
        float xa[8], xb[8];
        unpack8(x.a, xa);
        unpack8(x.b, xb);
        float ss = 0.f, hx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
          hx = fmaf(ga[e] * wa[e], xa[e], fmaf(gb[e] * wb[e], xb[e], hx));
        }
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        const float m = row_sum<LPR>(hx) * (1.f / D) * r;  // mean of h n
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float na = xa[e] * r, nb = xb[e] * r;
          dwa[e] = fmaf(ga[e], na, dwa[e]);
          dwb[e] = fmaf(gb[e], nb, dwb[e]);
          ga[e] = r * (ga[e] * wa[e] - na * m);
          gb[e] = r * (gb[e] * wb[e] - nb * m);
        }
      }
      if (live) store_row(dx_t, b * dx_t.sb + h * dx_t.sh + n * dx_t.sn, ln, ga, gb, err);
    }
  }
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        dwa[e] += __shfl_xor_sync(0xffffffffu, dwa[e], o);
        dwb[e] += __shfl_xor_sync(0xffffffffu, dwb[e], o);
      }
    }
    if ((threadIdx.x & 31) < LPR) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        red[threadIdx.x >> 5][ln.ca * 8 + e] = dwa[e];
        red[threadIdx.x >> 5][ln.cb * 8 + e] = dwb[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += red[w][threadIdx.x];
      const long long at = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x;
      if (in_range(at, 1, 2ll * gridDim.x * D, err)) partial[at] = s;
    }
  }
}

// dw = Σ of the CTAs' partial rows, in a fixed order and in 64 bits (a few
// hundred values a dimension: the partial rows' own rounding is what stays).
template <int D>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* __restrict__ partial, int n_parts,
                                                           float* __restrict__ dqw, float* __restrict__ dkw) {
  constexpr int SLICES = 1024 / D;
  uint32_t* err = &g_rope_err;
  __shared__ double red[SLICES][D];
  const int c = threadIdx.x % D, slice = threadIdx.x / D;
  double s = 0.0;
  for (int i = slice; i < n_parts; i += SLICES) {
    const long long at = (static_cast<long long>(blockIdx.x) * n_parts + i) * D + c;
    if (in_range(at, 1, 2ll * n_parts * D, err)) s += partial[at];
  }
  red[slice][c] = s;
  __syncthreads();
  if (slice == 0) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < SLICES; ++i) v += red[i][c];
    (blockIdx.x ? dkw : dqw)[c] = static_cast<float>(v);
  }
}

template <int D>
static cudaError_t fwd(NormRope p, cudaStream_t stream) {
  constexpr int ROWS = THREADS / (D / 16), HPG = 4;
  p.q_groups = (p.H + HPG - 1) / HPG;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const dim3 grid(static_cast<unsigned>((tokens + ROWS - 1) / ROWS),
                  static_cast<unsigned>(p.q_groups + (p.Hkv + HPG - 1) / HPG));
  norm_rope_kernel<D, HPG><<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t bwd(const NormRope& p, float* partial, int parts, float* dqw, float* dkw, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(parts), 2);
  if (!p.q_weight) {
    norm_rope_bwd_kernel<D, false><<<grid, THREADS, 0, stream>>>(p, nullptr);
    return cudaGetLastError();
  }
  norm_rope_bwd_kernel<D, true><<<grid, THREADS, 0, stream>>>(p, partial);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  weight_grad_kernel<D><<<2, 1024, 0, stream>>>(partial, parts, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace rope

int norm_rope_bwd_parts(int B, int N, int d) {
  const long long rows = rope::THREADS / (d / 16);
  const long long tiles = (static_cast<long long>(B) * N + rows - 1) / rows;
  return static_cast<int>(tiles < 304 ? tiles : 304);
}

cudaError_t launch_norm_rope(const NormRope& p, int d, cudaStream_t stream) {
  return d == 64 ? rope::fwd<64>(p, stream) : rope::fwd<128>(p, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRope& p, int d, float* partial, float* dqw, float* dkw,
                                 cudaStream_t stream) {
  const int parts = norm_rope_bwd_parts(p.B, p.N, d);
  return d == 64 ? rope::bwd<64>(p, partial, parts, dqw, dkw, stream)
                 : rope::bwd<128>(p, partial, parts, dqw, dkw, stream);
}

cudaError_t read_and_clear_rope_error(uint32_t* out, cudaStream_t stream) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_rope_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbolAsync(g_rope_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return e;
  return cudaStreamSynchronize(stream);
}

}  // namespace fa
