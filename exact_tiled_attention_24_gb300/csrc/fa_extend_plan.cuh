// How the work of a chunk call (fa_extend.cu) is cut into pieces: pure integer
// functions of the requests' lengths, evaluated by the attention kernel and by
// the merge, which must agree.
//
//   item    two query tiles of one K/V head of one request: up to 2·tpt new
//           tokens with the heads that share the K/V head (256 rows)
//   unit    one 128-key tile of one item, the work of one step of a CTA
//   order   request by request, (chunk,) K/V head, item, key tile. The units
//           in this order are cut into C equal shares, one a CTA: the lengths
//           are on the device only, and equal shares need no rule for uneven
//           ones. An item that crosses from one share to the next is finished
//           by a merge of its parts.
//   chunk   a request with several items reads its keys once an item. CTAs
//           with equal shares stand at different keys of it, so what one reads
//           has left L2 before another needs it. The keys are therefore cut
//           into chunks of `lc` tiles (their K and V fit L2), and all items
//           pass one chunk before any passes the next.
#pragma once

#include <cstdint>

#include "fa_common.h"
#include "fa_ptx.cuh"

#define FA_HD __host__ __device__ __forceinline__

namespace fa {
namespace ext {

constexpr int TK = 128;          // keys a tile
constexpr int MIN_SHARE = 4;     // units a CTA has at least
constexpr int MAX_CTAS = 152;
constexpr int SHARE_CHUNKS = 8;  // chunks are at least 1/8 of a share long

typedef unsigned long long u64;

// One request: its first row of q, new tokens, cached tokens, items.
struct Request {
  int row0, n, len, items;
  FA_HD int base() const { return len - n; }  // position of its first new token
};

__device__ __forceinline__ Request request_of(const Extend& p, int b, uint32_t* err) {
  Request r{0, 0, 0, 0};
  const int s = p.q_starts[b], e = p.q_starts[b + 1];
  if (s < 0 || e > p.T || e < s) {
    atomicExch(err, DEV_BAD_INDEX);
    return r;
  }
  r.row0 = s, r.n = e - s;
  r.len = min(max(p.seq_lens[b], 0), p.max_blocks * p.bs);
  r.items = (r.n + 2 * p.tpt - 1) / (2 * p.tpt);
  return r;
}

// Σ_{i < n} floor((a i + b) / m), by Euclid's steps (a and m below 2^9).
FA_HD u64 floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  u64 s = 0;
  while (n > 0) {
    if (a >= m) s += static_cast<u64>(n) * (n - 1) / 2 * (a / m), a %= m;
    if (b >= m) s += static_cast<u64>(n) * (b / m), b %= m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m, b = top % m;
    const uint32_t t = a;
    a = m, m = t;
  }
  return s;
}

struct Shape {
  int span;  // tokens an item: 2·tpt
  bool causal;
  int lc;    // key tiles a chunk

  FA_HD static int tiles_to(int keys) { return max(1, (max(keys, 0) + TK - 1) / TK); }
  // key tiles item i sees (one at least, so that its rows are written)
  FA_HD int tiles(const Request& r, int i) const {
    return tiles_to(causal ? r.base() + min((i + 1) * span, r.n) : r.len);
  }
  // Σ_{i' < i} tiles(i')
  FA_HD u64 before(const Request& r, int i) const {
    if (!causal) return static_cast<u64>(i) * tiles_to(r.len);
    const int full = min(i, r.items - 1);  // the last item may be shorter
    const int ones = min(full, r.base() >= TK ? 0 : (TK - r.base()) / span);
    u64 s = ones;
    if (full > ones) s += floor_sum(full - ones, TK, span, r.base() + (ones + 1) * span + TK - 1);
    return i > full ? s + tiles(r, i - 1) : s;
  }
  // the first item that sees more than x tiles
  FA_HD int past(const Request& r, long long x) const {
    if (x <= 0) return 0;
    if (static_cast<long long>(r.len) <= x * TK) return r.items;
    if (!causal) return 0;
    const long long d = x * TK - r.base();
    return d < 0 ? 0 : static_cast<int>(min(d / span, static_cast<long long>(r.items - 1)));
  }
  FA_HD bool chunked(const Request& r) const {
    return r.items > 1 && tiles(r, r.items - 1) > lc;
  }
  FA_HD int chunks(const Request& r) const {
    return chunked(r) ? (tiles(r, r.items - 1) + lc - 1) / lc : 1;
  }
  // tiles of item i in chunk c
  FA_HD int length(const Request& r, int c, int i) const {
    const int t = tiles(r, i);
    return chunked(r) ? min(max(t - c * lc, 0), lc) : t;
  }
  // Σ_{c' < c} of the tiles of one head in chunk c'
  FA_HD u64 chunks_before(const Request& r, int c) const {
    if (c == 0) return 0;
    const int i = past(r, static_cast<long long>(c) * lc);
    return before(r, i) + static_cast<u64>(r.items - i) * (static_cast<u64>(c) * lc);
  }
  // Σ_{i' < i} length(c, i')
  FA_HD u64 in_chunk_before(const Request& r, int c, int i) const {
    if (!chunked(r)) return before(r, i);
    const int i0 = past(r, static_cast<long long>(c) * lc), i1 = past(r, static_cast<long long>(c + 1) * lc);
    if (i <= i0) return 0;
    const int j = max(i0, min(i, i1));
    u64 s = before(r, j) - before(r, i0) - static_cast<u64>(j - i0) * (static_cast<u64>(c) * lc);
    if (i > j) s += static_cast<u64>(i - j) * lc;
    return s;
  }
  // Items that pass more than one chunk are "long"; each of their chunks has a
  // part of its own. The first long item that reaches chunk c:
  FA_HD int first_long(const Request& r, int c) const {
    return past(r, static_cast<long long>(max(c, 1)) * lc);
  }
  FA_HD bool is_long(const Request& r, int i) const { return chunked(r) && tiles(r, i) > lc; }
  // parts of one head's long items in the chunks before c
  FA_HD int long_before(const Request& r, int c) const {
    int s = 0;
    for (int x = 0; x < c; ++x) s += r.items - first_long(r, x);
    return s;
  }
};

// The whole call's cut. C shares of U units: share k is [start(k), start(k + 1)).
struct Cut {
  u64 units;
  int ctas;
  FA_HD u64 start(int k) const { return units * static_cast<u64>(k) / ctas; }
  FA_HD int owner(u64 u) const { return static_cast<int>(((u + 1) * ctas - 1) / units); }
};

// Where a unit lies, with what lies before its request.
struct Place {
  Request r;
  int b;
  u64 units0;  // units before the request
  int longs0;  // parts of long items before the request
  int c, hv, i;
  int off;     // tile of the item within the chunk
};

// Block-wide exclusive scan of one value a thread.
template <int NT>
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();  // the scratch may be in use
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  u64 below = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const u64 t = scratch[w];
    if (w < warp) below += t;
    all += t;
  }
  *total = all;
  return below + s - v;
}

struct PlanSmem {
  u64 scan[16];
  u64 units0, items0;
  int b, longs0;
};

__device__ __forceinline__ u64 units_of(const Extend& p, const Shape& sh, const Request& r) {
  return r.n > 0 ? sh.before(r, r.items) * p.hv : 0;
}

// The cut of the whole call (the shape's chunk length is set on the way).
template <int NT>
__device__ __forceinline__ Cut cut_of(const Extend& p, Shape* sh, PlanSmem* sm, uint32_t* err) {
  u64 mine = 0, total;
  for (int b = threadIdx.x; b < p.B; b += NT) mine += units_of(p, *sh, request_of(p, b, err));
  block_scan<NT>(mine, sm->scan, &total);
  Cut cut;
  cut.units = total;
  const u64 most = total / MIN_SHARE;
  cut.ctas = static_cast<int>(most < 1 ? 1 : most > static_cast<u64>(p.ctas) ? p.ctas : most);
  const u64 least = (total + SHARE_CHUNKS * cut.ctas - 1) / (SHARE_CHUNKS * cut.ctas);
  sh->lc = least > static_cast<u64>(p.lc) ? static_cast<int>(least) : p.lc;
  return cut;
}

// The request that holds unit `target` (LONG = false), or the target-th long
// item (LONG = true); found by one thread, known to all afterwards. Returns
// false if there is none.
template <int NT, bool LONG>
__device__ __forceinline__ bool find_request(const Extend& p, const Shape& sh, PlanSmem* sm, u64 target, Place* at,
                                             u64* items0, uint32_t* err) {
  if (threadIdx.x == 0) sm->b = -1;
  u64 units = 0, longs = 0, items = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    Request r{0, 0, 0, 0};
    if (b < p.B) r = request_of(p, b, err);
    const u64 u = units_of(p, sh, r);
    u64 l = 0, it = 0;
    if (p.may_chunk && r.n > 0 && sh.chunked(r)) {
      l = static_cast<u64>(sh.long_before(r, sh.chunks(r))) * p.hv;
      it = static_cast<u64>(r.items - sh.first_long(r, 0)) * p.hv;
    }
    u64 tu, tl = 0, ti = 0;
    const u64 eu = units + block_scan<NT>(u, sm->scan, &tu);
    u64 el = longs, ei = items;
    if (p.may_chunk) {
      el += block_scan<NT>(l, sm->scan, &tl);
      ei += block_scan<NT>(it, sm->scan, &ti);
    }
    const u64 key = LONG ? ei : eu, size = LONG ? it : u;
    if (target >= key && target - key < size) sm->b = b, sm->units0 = eu, sm->longs0 = static_cast<int>(el), sm->items0 = ei;
    units += tu, longs += tl, items += ti;
  }
  __syncthreads();
  at->b = sm->b;
  if (at->b < 0) return false;
  at->r = request_of(p, at->b, err);
  at->units0 = sm->units0;
  at->longs0 = sm->longs0;
  *items0 = sm->items0;
  return true;
}

// The rest of a unit's place within its request; run by a whole warp.
__device__ __forceinline__ void locate(const Extend& p, const Shape& sh, u64 u, Place* at) {
  const int lane = threadIdx.x & 31;
  const Request& r = at->r;
  u64 rem = u - at->units0;
  const int n_c = sh.chunks(r);
  int c = 0;
  for (int c0 = 0; c0 < n_c; c0 += 32) {
    const bool ok = c0 + lane < n_c && sh.chunks_before(r, c0 + lane) * p.hv <= rem;
    const int cnt = __popc(__ballot_sync(0xffffffffu, ok));
    if (cnt > 0) c = c0 + cnt - 1;
    if (cnt < 32) break;
  }
  rem -= sh.chunks_before(r, c) * p.hv;
  const u64 row = sh.in_chunk_before(r, c, r.items);
  at->c = c;
  at->hv = static_cast<int>(rem / row);
  rem -= row * at->hv;
  int lo = sh.chunked(r) ? sh.past(r, static_cast<long long>(c) * sh.lc) : 0, hi = r.items;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
    const bool ok = probe < hi && sh.in_chunk_before(r, c, probe) <= rem;
    const int cnt = __popc(__ballot_sync(0xffffffffu, ok));
    lo += (cnt - 1) * step;
    hi = min(hi, lo + step);
  }
  at->i = lo;
  at->off = static_cast<int>(rem - sh.in_chunk_before(r, c, lo));
}

// Where a piece's result goes: slots 2k and 2k + 1 are CTA k's first and last
// piece where its share cuts an item, the others hold whole chunks of long
// items; -1: the outputs themselves.
__device__ __forceinline__ int part_slot(const Extend& p, const Shape& sh, const Cut& cut, const Place& at, int k,
                                         bool start_cut, bool end_cut) {
  if (start_cut) return 2 * k;
  if (end_cut) return 2 * k + 1;
  if (!sh.is_long(at.r, at.i)) return -1;
  const int in_c = at.r.items - sh.first_long(at.r, at.c);
  return 2 * p.ctas + at.longs0 + p.hv * sh.long_before(at.r, at.c) + at.hv * in_c + at.i - sh.first_long(at.r, at.c);
}

}  // namespace ext
}  // namespace fa
