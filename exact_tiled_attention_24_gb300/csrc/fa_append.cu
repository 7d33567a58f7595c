// Appending new tokens' keys and values to a paged KV cache, with the norm
// and position rotation of keys (and of the tokens' queries) on the way, in
// bf16 or in 4-bit codes (fa_rope.cuh has one row's norm and rotation,
// fa_q4.cuh the codes).
//
// Token t belongs to request requests[t], at position positions[t] of it:
// that is its cache slot (block block_table[request][position / bs], slot
// position % bs) and the row of the rotation tables. It is one read and one
// write per element; a row of D / 16 lanes takes one head of one token.
//
// 16384 prompt tokens of 32 + 8 + 8 heads, d = 128: 70 us into a bf16 cache
// (86% of the measured copy rate), 86 us into 4-bit codes with the values held
// written beside them (73%: the integer pipe is at 46% then, DRAM at 59%, and
// neither is full: one body for queries, keys and values keeps weights, angles
// and four heads' loads, and spills 28 to 36 bytes a thread). A
// decode step of 32 tokens takes 6 to 7 us, a chain of dependent loads
// (position, block table, angles) and one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"
#include "fa_q4.cuh"
#include "fa_rope.cuh"

namespace fa {

static __device__ uint32_t g_append_err;

namespace append {

constexpr int THREADS = 128;

using rope::Angles;
using rope::Lane;
using rope::Raw;
using rope::Row;

// Which rows a group of heads holds.
enum Part : int { QUERIES = 0, KEYS = 1, VALUES = 2 };

__device__ __forceinline__ Raw load_row(const TokenRows& t, long long off, const Lane& ln, uint32_t* err) {
  Raw r{};
  if (in_range(off + ln.ca * 8, 8, t.extent, err)) r.a = rope::load16(t.p + off + ln.ca * 8);
  if (in_range(off + ln.cb * 8, 8, t.extent, err)) r.b = rope::load16(t.p + off + ln.cb * 8);
  return r;
}

__device__ __forceinline__ void store_chunks(__nv_bfloat16* base, long long extent, long long off, const Lane& ln,
                                             const Row& x, uint32_t* err) {
  if (in_range(off + ln.ca * 8, 8, extent, err)) rope::store16(base + off + ln.ca * 8, rope::pack8(x.a));
  if (in_range(off + ln.cb * 8, 8, extent, err)) rope::store16(base + off + ln.cb * 8, rope::pack8(x.b));
}

// Where token t goes: its position and cache block, or live = false for a
// padding token (negative request or position) and for one whose request,
// position or block lies outside what the caller gave (reported).
struct Slot {
  bool live;
  int pos, block;
};
template <bool AXES>
__device__ __forceinline__ Slot slot_of(const Append& p, long long t, uint32_t* err) {
  Slot s{false, 0, 0};
  if (t >= p.T || !in_range(t, 1, p.T, err)) return s;
  const int req = p.requests ? p.requests[t] : static_cast<int>(t);
  const int pos = p.positions[t];
  if (req < 0 || pos < 0) return s;
  if (req < p.B && pos / p.bs < p.max_blocks && (AXES || p.rot == 0 || pos < p.n_pos)) {
    const long long ti = static_cast<long long>(req) * p.max_blocks + pos / p.bs;
    const int blk = in_range(ti, 1, static_cast<long long>(p.B) * p.max_blocks, err) ? p.block_table[ti] : -1;
    if (blk >= 0 && blk < p.num_blocks) return Slot{true, pos, blk};
  }
  atomicExch(err, DEV_BAD_INDEX);
  return s;
}

// A row of lanes takes one token and a section of the heads of its queries,
// keys or values (blockIdx.y says which), two heads at a time with the next
// two on their way.
constexpr int STEP = 2;
template <int D, bool Q4, bool INTER, bool AXES>
__global__ void __launch_bounds__(THREADS, 5) append_kernel(const Append p) {
  constexpr int LPR = D / 16, ROWS = THREADS / LPR, NG = D / 64;
  uint32_t* err = &g_append_err;
  const int i = threadIdx.x % LPR;
  const long long t = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / LPR;
  int sec = static_cast<int>(blockIdx.y);
  const int part = sec < p.q_sections ? QUERIES : sec < p.q_sections + p.kv_sections ? KEYS : VALUES;
  sec -= part == QUERIES ? 0 : part == KEYS ? p.q_sections : p.q_sections + p.kv_sections;
  const int n_sec = part == QUERIES ? p.q_sections : p.kv_sections, heads = part == QUERIES ? p.H : p.Hkv;
  const int h0 = static_cast<int>(static_cast<long long>(sec) * heads / n_sec);  // sections as even as they go
  const int h1 = static_cast<int>(static_cast<long long>(sec + 1) * heads / n_sec);
  const TokenRows& src = part == QUERIES ? p.q : part == KEYS ? p.k : p.v;
  const Lane ln(i, part == VALUES ? 0 : p.rot);
  auto load = [&](int h, Raw (&r)[STEP]) {
#pragma unroll
    for (int j = 0; j < STEP; ++j)
      r[j] = t < p.T && h + j < h1 ? load_row(src, t * src.st + (h + j) * src.sh, ln, err) : Raw{};
  };
  Raw cur[STEP], next[STEP];
  load(h0, cur);
  Slot slot = slot_of<AXES>(p, t, err);
  Angles ang;
  bool turned = part != VALUES && ln.turned && slot.live;
  if constexpr (AXES) {  // the rotary positions are apart from the slot, and as much as the slot what makes a token live
    const rope::AxisRows rows(p.axes, slot.live ? t : 0, p.n_pos, err);
    if (slot.live && !rows.ok) {
      atomicExch(err, DEV_BAD_INDEX);
      slot.live = turned = false;
    }
    if (turned) ang.load(p.cos, p.sin, rows, p.axes, p.rot, ln, INTER);
  } else if (turned) {
    ang.load(p.cos, p.sin, slot.pos, p.rot, ln, INTER);
  }
  const void* w = part == QUERIES ? p.q_weight : part == KEYS ? p.k_weight : nullptr;
  Row wt;
  if (w) {
    rope::load_weight8(w, p.w32, ln.ca, wt.a);
    rope::load_weight8(w, p.w32, ln.cb, wt.b);
  }
  // the cache's row of the token's slot in K/V head 0
  const long long row0 = static_cast<long long>(slot.block) * p.Hkv * p.bs + slot.pos % p.bs;
  const long long rows = static_cast<long long>(p.num_blocks) * p.Hkv * p.bs;
  for (int hh = h0; hh < h1; hh += STEP) {
    load(hh + STEP, next);
  #pragma unroll
    for (int j = 0; j < STEP; ++j) {
      Row x = rope::unpack(cur[j]);
      cur[j] = next[j];
      const int h = hh + j;
      if (w) x = rope::times(rope::times(x, rope::inv_rms<LPR>(x, p.eps)), wt);
      if (turned) rope::turn<false>(x, ang, INTER);
      const bool mine = slot.live && h < h1;
      if (part == QUERIES) {
        const long long at = t * p.q_out.st + h * p.q_out.sh;
        if (mine) store_chunks(p.q_out.p, p.q_out.extent, at, ln, x, err);
        else if (p.zero_skipped && t < p.T && h < h1) store_chunks(p.q_out.p, p.q_out.extent, at, ln, Row{}, err);
        continue;
      }
      const long long row = row0 + static_cast<long long>(h) * p.bs;
      if (!Q4) {
        if (mine)
          store_chunks(static_cast<__nv_bfloat16*>(part == KEYS ? p.k_cache : p.v_cache), rows * D, row * D, ln, x,
                       err);
        continue;
      }
      q4::Grid grid[NG];
      q4::grids<D>(x, ln, i, grid);
      if (mine) {
        uint8_t* codes = static_cast<uint8_t*>(part == KEYS ? p.k_cache : p.v_cache);
        __nv_bfloat16* pairs = part == KEYS ? p.k_scale : p.v_scale;
        const q4::Grid ga = NG == 1 || ln.ca / 8 == 0 ? grid[0] : grid[NG - 1];
        const q4::Grid gb = NG == 1 || ln.cb / 8 == 0 ? grid[0] : grid[NG - 1];
        Row n;
        const uint32_t wa4 = q4::encode8(x.a, ga, n.a), wb4 = q4::encode8(x.b, gb, n.b);
        if (in_range(row * (D / 2) + ln.ca * 4, 4, rows * (D / 2), err))
          *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + ln.ca * 4) = wa4;
        if (in_range(row * (D / 2) + ln.cb * 4, 4, rows * (D / 2), err))
          *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + ln.cb * 4) = wb4;
        const int own = q4::own_group<D>(i);
        if (i % (LPR / NG) == 0 && in_range((row * NG + own) * 2, 2, rows * NG * 2, err))
          *reinterpret_cast<uint32_t*>(pairs + (row * NG + own) * 2) = q4::pair(grid[own]);
        __nv_bfloat16* held = part == KEYS ? p.k_values : p.v_values;
        if (held) {
          q4::held8(n.a, ga, x.a);
          q4::held8(n.b, gb, x.b);
          store_chunks(held, static_cast<long long>(p.T) * p.Hkv * D, (t * p.Hkv + h) * D, ln, x, err);
        }
      }
    }
  }
}

template <int D, bool Q4>
static cudaError_t launch(Append p, cudaStream_t stream) {
  constexpr int ROWS = THREADS / (D / 16);
  const long long tiles = (p.T + ROWS - 1) / ROWS;
  // Sections of up to 16 heads, smaller ones until a wave of CTAs is there.
  for (int hs = 16; hs > 1; hs /= 2) {
    p.q_sections = (p.H + hs - 1) / hs;
    p.kv_sections = (p.Hkv + hs - 1) / hs;
    if (tiles * (p.q_sections + 2 * p.kv_sections) >= 152 * 5) break;
  }
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.q_sections + 2 * p.kv_sections));
  const auto kern = p.axes.n > 0 ? (p.interleaved ? append_kernel<D, Q4, true, true> : append_kernel<D, Q4, false, true>)
                                 : (p.interleaved ? append_kernel<D, Q4, true, false> : append_kernel<D, Q4, false, false>);
  kern<<<grid, THREADS, 0, stream>>>(p);
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
