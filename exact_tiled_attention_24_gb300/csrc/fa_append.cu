// Appending new tokens' keys and values to a paged KV cache, with the norm
// and position rotation of keys (and of the tokens' queries) on the way, in
// bf16 or in 4-bit codes (fa_rope.cuh has one row's norm and rotation,
// fa_q4.cuh the codes).
//
// Token t belongs to request requests[t], at position positions[t] of it:
// that is its cache slot (block block_table[request][position / bs], slot
// position % bs) and the row of the rotation tables. It is one read and one
// write per element; a row of D / 16 lanes takes one head of one token.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_q4.cuh"
#include "fa_rope.cuh"

namespace fa {

static __device__ uint32_t g_append_err;

namespace append {

constexpr int THREADS = 256;

using rope::Angles;
using rope::Lane;
using rope::Raw;

// Which rows a group of heads holds.
enum Part : int { QUERIES = 0, KEYS = 1, VALUES = 2 };

__device__ __forceinline__ Raw load_row(const TokenRows& t, long long off, const Lane& ln, uint32_t* err) {
  Raw r{};
  if (in_range(off + ln.ca * 8, 8, t.extent, err)) r.a = *reinterpret_cast<const uint4*>(t.p + off + ln.ca * 8);
  if (in_range(off + ln.cb * 8, 8, t.extent, err)) r.b = *reinterpret_cast<const uint4*>(t.p + off + ln.cb * 8);
  return r;
}

__device__ __forceinline__ void store_chunks(__nv_bfloat16* base, long long extent, long long off, const Lane& ln,
                                             const float* a, const float* b, uint32_t* err) {
  if (in_range(off + ln.ca * 8, 8, extent, err)) *reinterpret_cast<uint4*>(base + off + ln.ca * 8) = rope::pack8(a);
  if (in_range(off + ln.cb * 8, 8, extent, err)) *reinterpret_cast<uint4*>(base + off + ln.cb * 8) = rope::pack8(b);
}

// Where token t goes: its position and cache block, or live = false for a
// padding token (negative request or position) and for one whose request,
// position or block lies outside what the caller gave (reported).
struct Slot {
  bool live;
  int pos, block;
};
__device__ __forceinline__ Slot slot_of(const Append& p, long long t, uint32_t* err) {
  Slot s{false, 0, 0};
  if (t >= p.T || !in_range(t, 1, p.T, err)) return s;
  const int req = p.requests ? p.requests[t] : static_cast<int>(t);
  const int pos = p.positions[t];
  if (req < 0 || pos < 0) return s;
  if (req < p.B && pos / p.bs < p.max_blocks && (p.rot == 0 || pos < p.n_pos)) {
    const long long ti = static_cast<long long>(req) * p.max_blocks + pos / p.bs;
    const int blk = in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err) ? p.block_table[ti] : -1;
    if (blk >= 0 && blk < p.num_blocks) return Slot{true, pos, blk};
  }
  atomicExch(err, DEV_BAD_INDEX);
  return s;
}

template <int D, int HPG, bool Q4>
__global__ void __launch_bounds__(THREADS) append_kernel(const Append p) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR, NG = D / 64;
  uint32_t* err = &g_append_err;
  const int i = threadIdx.x % LPR;
  const long long t = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / LPR;
  int group = static_cast<int>(blockIdx.y);
  const int part = group < p.q_groups ? QUERIES : group < p.q_groups + p.kv_groups ? KEYS : VALUES;
  group -= part == QUERIES ? 0 : part == KEYS ? p.q_groups : p.q_groups + p.kv_groups;
  const int h0 = group * HPG;
  const int heads = min(HPG, (part == QUERIES ? p.H : p.Hkv) - h0);
  const TokenRows& src = part == QUERIES ? p.q : part == KEYS ? p.k : p.v;
  const Lane ln(i, part == VALUES ? 0 : p.rot);

  Raw raw[HPG];
#pragma unroll
  for (int j = 0; j < HPG; ++j)
    raw[j] = t < p.T && j < heads ? load_row(src, t * src.st + (h0 + j) * src.sh, ln, err) : Raw{};
  const Slot slot = slot_of(p, t, err);
  Angles ang;
  const bool turned = part != VALUES && ln.turned && slot.live;
  if (turned) ang.load(p.cos, p.sin, slot.pos, p.rot, ln, p.interleaved);
  const void* w = part == QUERIES ? p.q_weight : part == KEYS ? p.k_weight : nullptr;
  float wa[8], wb[8];
  if (w) {
    rope::load_weight8(w, p.w32, ln.ca, wa);
    rope::load_weight8(w, p.w32, ln.cb, wb);
  }
  const int in_block = slot.pos % p.bs;
#pragma unroll
  for (int j = 0; j < HPG; ++j) {
    float a[8], c[8];
    rope::unpack8(raw[j].a, a);
    rope::unpack8(raw[j].b, c);
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(c[e], c[e], ss));
      const float r = rsqrtf(rope::row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * r * wa[e];
        c[e] = c[e] * r * wb[e];
      }
    }
    if (turned) rope::turn(a, c, ang, p.interleaved, 1.f);
    const bool mine = slot.live && j < heads;
    const int h = h0 + j;
    if (part == QUERIES) {
      if (mine) store_chunks(p.q_out.p, p.q_out.extent, t * p.q_out.st + h * p.q_out.sh, ln, a, c, err);
      continue;
    }
    // row of the cache: block, K/V head, slot
    const long long row = (static_cast<long long>(slot.block) * p.Hkv + h) * p.bs + in_block;
    const long long rows = static_cast<long long>(p.num_blocks) * p.Hkv * p.bs;
    if (!Q4) {
      if (mine)
        store_chunks(static_cast<__nv_bfloat16*>(part == KEYS ? p.k_cache : p.v_cache), rows * D, row * D, ln, a, c,
                     err);
      continue;
    }
    q4::Grid grid[NG];
    q4::grids<D>(a, c, ln, grid);
    if (mine) {
      uint8_t* codes = static_cast<uint8_t*>(part == KEYS ? p.k_cache : p.v_cache);
      __nv_bfloat16* pairs = part == KEYS ? p.k_scale : p.v_scale;
      const q4::Grid ga = grid[NG == 1 ? 0 : ln.ca / 8], gb = grid[NG == 1 ? 0 : ln.cb / 8];
      const uint32_t wa4 = q4::encode8(a, ga), wb4 = q4::encode8(c, gb);
      if (in_range(row * (D / 2) + ln.ca * 4, 4, rows * (D / 2), err))
        *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + ln.ca * 4) = wa4;
      if (in_range(row * (D / 2) + ln.cb * 4, 4, rows * (D / 2), err))
        *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + ln.cb * 4) = wb4;
      if (i < NG && in_range((row * NG + i) * 2, 2, rows * NG * 2, err))
        *reinterpret_cast<uint32_t*>(pairs + (row * NG + i) * 2) = q4::pair(grid[NG == 1 ? 0 : i]);
      __nv_bfloat16* held = part == KEYS ? p.k_values : p.v_values;
      if (held) {
        q4::decode8(wa4, ga, a);
        q4::decode8(wb4, gb, c);
        store_chunks(held, static_cast<long long>(p.T) * p.Hkv * D, (t * p.Hkv + h) * D, ln, a, c, err);
      }
    }
  }
}

template <int D, bool Q4>
static cudaError_t launch(Append p, cudaStream_t stream) {
  constexpr int ROWS = THREADS / (D / 16), HPG = 4;
  p.q_groups = (p.H + HPG - 1) / HPG;
  p.kv_groups = (p.Hkv + HPG - 1) / HPG;
  const dim3 grid(static_cast<unsigned>((p.T + ROWS - 1) / ROWS), static_cast<unsigned>(p.q_groups + 2 * p.kv_groups));
  append_kernel<D, HPG, Q4><<<grid, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace append

cudaError_t launch_append(const Append& p, int d, bool q4, cudaStream_t stream) {
  if (d == 64) return q4 ? append::launch<64, true>(p, stream) : append::launch<64, false>(p, stream);
  return q4 ? append::launch<128, true>(p, stream) : append::launch<128, false>(p, stream);
}

cudaError_t read_and_clear_append_error(uint32_t* out, cudaStream_t stream) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_append_err, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbolAsync(g_append_err, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return e;
  return cudaStreamSynchronize(stream);
}

}  // namespace fa
