// Per-head norms of q and k with the position rotation in the same pass, and
// their gradient: what stands between a layer's projections and the
// attention forward (fa_rope.cuh has the formulas of one row).
//
// Gradient of one row for the output gradient dy, with g = Rᵀ dy (the
// rotation turned back), n = x r (the normed row) and h = g w:
//     dx = r (h − n · mean_c(h_c n_c)),     dw = Σ_rows g n.
// x is read again and r formed again from it: saving r would cost a write
// and a read of 4 bytes per row against nothing but a sum.
//
// Both are bound by memory: one read and one write per element (the gradient
// two reads). Measured for B = 2, 32 + 8 heads, N = 8192, d = 128: forward
// 58 us (its 340 MB at 86% of the measured copy rate), gradient 95 us (507 MB,
// 79%; its loads in flight are limited by registers).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_rope.cuh"

namespace fa {

static __device__ uint32_t g_rope_err;

namespace rope {

constexpr int THREADS = 128;

// A lane's place in the rows of one token, moved from head to head: the
// address of its chunk a; chunk b is a fixed distance on.
struct Cursor {
  __nv_bfloat16* at;
  long long step;  // one head
  int to_b;        // chunk a to chunk b
  const HeadRows* t;
  __device__ __forceinline__ Cursor(const HeadRows& rows, int b, int n, int h, const Lane& ln)
      : at(rows.p + (b * rows.sb + n * rows.sn + h * rows.sh + ln.ca * 8)),
        step(rows.sh), to_b((ln.cb - ln.ca) * 8), t(&rows) {}
  __device__ __forceinline__ bool fits(const __nv_bfloat16* p, uint32_t* err) const {
    return in_range(p - t->p, 8, t->extent, err);
  }
  __device__ __forceinline__ Raw load(uint32_t* err) const {
    Raw r{};
    if (fits(at, err)) r.a = load16(at);
    if (fits(at + to_b, err)) r.b = load16(at + to_b);
    return r;
  }
  __device__ __forceinline__ void store(const Row& x, uint32_t* err) const {
    if (fits(at, err)) store16(at, pack8(x.a));
    if (fits(at + to_b, err)) store16(at + to_b, pack8(x.b));
  }
};

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

// The token's angles, and whether it has any (false: reported). AXES: of its
// positions on several axes.
template <bool AXES>
__device__ __forceinline__ bool angles_of(const NormRope& p, int b, int n, const Lane& ln, bool inter, Angles* t,
                                          uint32_t* err) {
  if constexpr (AXES) {
    const AxisRows rows(p.axes, b * p.pos_sb + n, p.n_pos, err);
    if (!rows.ok) atomicExch(err, DEV_BAD_INDEX);
    else if (ln.turned) t->load(p.cos, p.sin, rows, p.axes, p.rot, ln, inter);
    return rows.ok;
  } else {
    const int pos = position_of(p, b, n, err);
    if (ln.turned && pos >= 0) t->load(p.cos, p.sin, pos, p.rot, ln, inter);
    return pos >= 0;
  }
}

// Token `tok` of all B·N, split into batch and position in it.
struct Token {
  bool live;
  int b, n;
  __device__ __forceinline__ Token(const NormRope& p, long long tok) {
    live = tok < static_cast<long long>(p.B) * p.N;
    b = live ? static_cast<int>(static_cast<uint32_t>(tok) / static_cast<uint32_t>(p.N)) : 0;
    n = live ? static_cast<int>(tok - static_cast<long long>(b) * p.N) : 0;
  }
};

// Heads of section i of n, as even as they go.
__device__ __forceinline__ int section_start(int i, int n, int heads) {
  return static_cast<int>(static_cast<unsigned long long>(static_cast<uint32_t>(i)) * static_cast<uint32_t>(heads) /
                          static_cast<uint32_t>(n));
}

// Forward. A row of lanes takes one token and a section of the heads of q or
// of k (blockIdx.y says which), two heads at a time with the next two on
// their way: the token's angles and the weights are read once for the
// section. The rows of a warp are consecutive tokens, contiguous in the
// output. Five CTAs an SM (the case above: 58 us; four 62, six, with spilled
// registers, 68).
template <int D, bool INTER, bool AXES>
__global__ void __launch_bounds__(THREADS, 5) norm_rope_kernel(const NormRope p) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR;
  uint32_t* err = &g_rope_err;
  const Lane ln(threadIdx.x % LPR, p.rot);
  const Token tk(p, static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / LPR);
  const bool is_k = static_cast<int>(blockIdx.y) >= p.q_sections;
  const int sec = static_cast<int>(blockIdx.y) - (is_k ? p.q_sections : 0);
  const int n_sec = is_k ? p.k_sections : p.q_sections, heads = is_k ? p.Hkv : p.H;
  const int h0 = section_start(sec, n_sec, heads), h1 = section_start(sec + 1, n_sec, heads);
  const HeadRows& src = is_k ? p.k : p.q;
  const HeadRows& dst = is_k ? p.k_out : p.q_out;
  Cursor in(src, tk.b, tk.n, h0, ln), out(dst, tk.b, tk.n, h0, ln);
  auto load2 = [&](int h, Raw (&r)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r[j] = tk.live && h + j < h1 ? in.load(err) : Raw{};
      in.at += in.step;
    }
  };
  Raw cur[2], next[2];
  load2(h0, cur);
  Angles t;
  const bool placed = tk.live && angles_of<AXES>(p, tk.b, tk.n, ln, INTER, &t, err);
  Row wt;
  const void* w = is_k ? p.k_weight : p.q_weight;
  if (w) {
    load_weight8(w, p.w32, ln.ca, wt.a);
    load_weight8(w, p.w32, ln.cb, wt.b);
  }
  for (int h = h0; h < h1; h += 2) {
    load2(h + 2, next);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      Row x = unpack(cur[j]);
      if (w) x = times(times(x, inv_rms<LPR>(x, p.eps)), wt);
      if (ln.turned && placed) turn<false>(x, t, INTER);
      if (!placed) x = Row{};  // no angle to turn by: a zero row
      if (tk.live && h + j < h1) out.store(x, err);
      out.at += out.step;
      cur[j] = next[j];
    }
  }
}

// Backward. The first parts_q CTAs take q, the others k. A CTA walks over
// items (a row of lanes' token, a section of the heads) of its tensor with
// its lanes' 16 dimensions of dw in registers and the next row on its way,
// then sums them over its rows in a fixed order into one partial row.
// Five CTAs an SM leave 96 registers a thread, and with a norm 72 to 104 bytes
// a thread are spilled; still 95 us (four CTAs and 608 parts: 103).
constexpr int MAX_PARTS = 760;
template <int D, bool NORM, bool INTER, bool AXES>
__global__ void __launch_bounds__(THREADS, 5) norm_rope_bwd_kernel(const NormRope p, int parts_q,
                                                                   float* __restrict__ partial) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR, WARPS = THREADS / 32;
  uint32_t* err = &g_rope_err;
  __shared__ float red[WARPS][D];
  __shared__ __align__(16) float weight[D];
  const bool is_k = static_cast<int>(blockIdx.x) >= parts_q;
  const int part = static_cast<int>(blockIdx.x) - (is_k ? parts_q : 0);
  const int parts = is_k ? static_cast<int>(gridDim.x) - parts_q : parts_q;
  const HeadRows& x_t = is_k ? p.k : p.q;
  const HeadRows& dy_t = is_k ? p.k_out : p.q_out;
  const HeadRows& dx_t = is_k ? p.dk : p.dq;
  const int heads = is_k ? p.Hkv : p.H;
  const int sections = is_k ? p.k_sections : p.q_sections;
  const Lane ln(threadIdx.x % LPR, p.rot);
  Row dw{};
  // The weights stay in shared memory (registers are what limits the CTAs an
  // SM), quarter by quarter of a lane's 16, so that a row's lanes read
  // consecutive 16 bytes.
  if constexpr (NORM) {
    const void* w = is_k ? p.k_weight : p.q_weight;
    for (int i = threadIdx.x; i < D; i += THREADS) {
      const Lane of((i / 4) % LPR, p.rot);
      const int quarter = i / (4 * LPR);
      const int c = (quarter < 2 ? of.ca : of.cb) * 8 + (quarter & 1) * 4 + i % 4;
      weight[i] = p.w32 ? reinterpret_cast<const float*>(w)[c]
                        : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c]);
    }
    __syncthreads();
  }
  const float* my_weight = weight + (threadIdx.x % LPR) * 4;
  const long long tiles = (static_cast<long long>(p.B) * p.N + ROWS - 1) / ROWS;
  for (long long item = part; item < tiles * sections; item += parts) {
    const int sec = static_cast<int>(item / tiles);
    const Token tk(p, (item - sec * tiles) * ROWS + threadIdx.x / LPR);
    const int h0 = section_start(sec, sections, heads), h1 = section_start(sec + 1, sections, heads);
    Cursor dy_at(dy_t, tk.b, tk.n, h0, ln), x_at(x_t, tk.b, tk.n, h0, ln), dx_at(dx_t, tk.b, tk.n, h0, ln);
    auto load = [&](int h, Raw& dy, Raw& x) {
      dy = x = Raw{};
      if (!tk.live || h >= h1) return;
      dy = dy_at.load(err);
      if (NORM) x = x_at.load(err);
      dy_at.at += dy_at.step;
      x_at.at += x_at.step;
    };
    Raw dy, x, dy_next, x_next;
    load(h0, dy, x);
    Angles t;
    const bool placed = tk.live && angles_of<AXES>(p, tk.b, tk.n, ln, INTER, &t, err);
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      load(h + 1, dy_next, x_next);
      Row g = unpack(dy);
      if (ln.turned && placed) turn<true>(g, t, INTER);
      // A row past the last token, or whose position the tables do not have
      // (the forward wrote zeros), adds nothing to dw and has no gradient. Ones
      // in place of x: a row of zeros has no finite r at eps = 0, and what the
      // input holds there may be NaN.
      if (!placed) {
        g = Row{};
        x.a = x.b = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
      }
      if (NORM) {
        // The sums first, then x unpacked and the weights read anew for the
        // rest: at 96 registers a thread they cannot stay.
        float r, m;
        {
          const Row xr = unpack(x), wt = shared_row<4 * LPR>(my_weight);
          r = inv_rms<LPR>(xr, p.eps);
          m = row_sum<LPR>(dot(times(g, wt), xr)) * (1.f / D) * r;  // mean of h n
        }
        forget(x);
        const float2 r2 = make_float2(r, r), rm = make_float2(-r * m, -r * m);
        auto rest = [&](float2& gv, float2& dwv, float2 xv, float2 wv) {
          const float2 nv = fmul2(xv, r2);
          dwv = ffma2(gv, nv, dwv);
          gv = ffma2(fmul2(gv, wv), r2, fmul2(nv, rm));  // r (h − n m)
        };
        const Row wt = shared_row<4 * LPR>(my_weight);
        const uint32_t xa[4] = {x.a.x, x.a.y, x.a.z, x.a.w}, xb[4] = {x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rest(g.a[e], dw.a[e], bf_pair(xa[e]), wt.a[e]);
          rest(g.b[e], dw.b[e], bf_pair(xb[e]), wt.b[e]);
        }
      }
      if (tk.live) dx_at.store(g, err);
      dx_at.at += dx_at.step;
      dy = dy_next;
      x = x_next;
    }
  }
  if constexpr (NORM) {
    launch_dependents();  // the sum over the CTAs may be set up; it waits for all of this grid's writes
    auto over_rows = [](float2& v) {  // Σ over the warp's rows
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      over_rows(dw.a[e]);
      over_rows(dw.b[e]);
    }
    if ((threadIdx.x & 31) < LPR) {
      float* mine = red[threadIdx.x >> 5];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2*>(mine + ln.ca * 8 + 2 * e) = dw.a[e];
        *reinterpret_cast<float2*>(mine + ln.cb * 8 + 2 * e) = dw.b[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += red[w][threadIdx.x];
      const long long at = static_cast<long long>(blockIdx.x) * D + threadIdx.x;
      if (in_range(at, 1, static_cast<long long>(gridDim.x) * D, err)) partial[at] = s;
    }
  }
}

// dw = Σ of the CTAs' partial rows, in a fixed order and in 64 bits (a few
// hundred values a dimension: the partial rows' own rounding is what stays).
// A CTA takes 8 dimensions, a thread every 32nd partial row of one.
constexpr int DW_COLS = 8, DW_SLICES = 32;
template <int D>
__global__ void __launch_bounds__(DW_COLS * DW_SLICES) weight_grad_kernel(const float* __restrict__ partial,
                                                                          int parts_q, int parts_k,
                                                                          float* __restrict__ dqw,
                                                                          float* __restrict__ dkw) {
  uint32_t* err = &g_rope_err;
  __shared__ double red[DW_SLICES][DW_COLS];
  const int c = threadIdx.x % DW_COLS, slice = threadIdx.x / DW_COLS;
  const int col = blockIdx.x * DW_COLS + c;
  const int n_parts = blockIdx.y ? parts_k : parts_q;
  wait_for_primary();
  const float* mine = partial + (blockIdx.y ? parts_q : 0) * D + col;
  double s = 0.0;
#pragma unroll 8
  for (int i = slice; i < n_parts; i += DW_SLICES)
    if (in_range(static_cast<long long>(i) * D + col, 1, static_cast<long long>(n_parts) * D, err))
      s += mine[static_cast<long long>(i) * D];
  red[slice][c] = s;
  __syncthreads();
  if (slice == 0) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < DW_SLICES; ++i) v += red[i][c];
    (blockIdx.y ? dkw : dqw)[col] = static_cast<float>(v);
  }
}

static void set_sections(NormRope* p, int hs) {
  p->q_sections = (p->H + hs - 1) / hs;
  p->k_sections = (p->Hkv + hs - 1) / hs;
}

template <int D>
static cudaError_t fwd(NormRope p, cudaStream_t stream) {
  constexpr int ROWS = THREADS / (D / 16);
  const long long tiles = (static_cast<long long>(p.B) * p.N + ROWS - 1) / ROWS;
  // Sections of up to 16 heads, smaller ones until a wave of CTAs is there.
  set_sections(&p, 16);
  for (int hs = 8; hs > 1 && tiles * (p.q_sections + p.k_sections) < 152 * 5; hs /= 2) set_sections(&p, hs);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.q_sections + p.k_sections));
  const auto kern = p.axes.n > 0 ? (p.interleaved ? norm_rope_kernel<D, true, true> : norm_rope_kernel<D, false, true>)
                                 : (p.interleaved ? norm_rope_kernel<D, true, false> : norm_rope_kernel<D, false, false>);
  kern<<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
static cudaError_t bwd(NormRope p, float* partial, float* dqw, float* dkw, cudaStream_t stream) {
  constexpr int ROWS = THREADS / (D / 16);
  const long long tiles = (static_cast<long long>(p.B) * p.N + ROWS - 1) / ROWS;
  // Sections of up to 8 heads; smaller ones while all items still fit one
  // wave (a second, part-filled one costs more than longer items).
  set_sections(&p, 8);
  for (int hs = 4; hs > 0; hs /= 2) {
    NormRope finer = p;
    set_sections(&finer, hs);
    if (tiles * (finer.q_sections + finer.k_sections) > MAX_PARTS) break;
    p = finer;
  }
  const long long items_q = tiles * p.q_sections, items_k = tiles * p.k_sections;
  // CTAs in proportion to the rows, at most as many as there are items
  long long parts_k = static_cast<long long>(MAX_PARTS) * p.Hkv / (p.H + p.Hkv);
  parts_k = parts_k < 1 ? 1 : parts_k > items_k ? items_k : parts_k;
  long long parts_q = MAX_PARTS - parts_k;
  parts_q = parts_q > items_q ? items_q : parts_q;
  if (items_q + items_k <= MAX_PARTS) parts_q = items_q, parts_k = items_k;
  const unsigned grid = static_cast<unsigned>(parts_q + parts_k);
  const bool norm = p.q_weight != nullptr;
  auto rows = [&](auto kern) { kern<<<grid, THREADS, 0, stream>>>(p, static_cast<int>(parts_q), norm ? partial : nullptr); };
  if (p.axes.n > 0) {
    if (norm) rows(p.interleaved ? norm_rope_bwd_kernel<D, true, true, true> : norm_rope_bwd_kernel<D, true, false, true>);
    else rows(p.interleaved ? norm_rope_bwd_kernel<D, false, true, true> : norm_rope_bwd_kernel<D, false, false, true>);
  } else {
    if (norm) rows(p.interleaved ? norm_rope_bwd_kernel<D, true, true, false> : norm_rope_bwd_kernel<D, true, false, false>);
    else rows(p.interleaved ? norm_rope_bwd_kernel<D, false, true, false> : norm_rope_bwd_kernel<D, false, false, false>);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !norm) return e;
  // Launched while the rows' kernel drains (4112 tokens of 12 + 12 heads, d =
  // 64: 16.7 us instead of 18.5).
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(D / DW_COLS, 2);
  cfg.blockDim = dim3(DW_COLS * DW_SLICES);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weight_grad_kernel<D>, static_cast<const float*>(partial), static_cast<int>(parts_q),
                            static_cast<int>(parts_k), dqw, dkw);
}

}  // namespace rope

size_t norm_rope_bwd_partial_bytes(int d) { return static_cast<size_t>(rope::MAX_PARTS) * d * sizeof(float); }

cudaError_t launch_norm_rope(const NormRope& p, int d, cudaStream_t stream) {
  return d == 64 ? rope::fwd<64>(p, stream) : rope::fwd<128>(p, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRope& p, int d, float* partial, float* dqw, float* dkw,
                                 cudaStream_t stream) {
  return d == 64 ? rope::bwd<64>(p, partial, dqw, dkw, stream) : rope::bwd<128>(p, partial, dqw, dkw, stream);
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
