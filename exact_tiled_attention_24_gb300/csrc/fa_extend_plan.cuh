// How the work of a chunk call (fa_extend.cu) is cut into pieces: pure integer
// functions of the requests' lengths, evaluated by the attention kernel and by
// the merge, which must agree. (tests/test_extend_plan.py evaluates them on the
// host, beside an enumeration.)
//
//   request one whose rows overlap those of an earlier one, or lie before them,
//           is taken for empty (Request::behind)
//   item    two query tiles of one K/V head of one request: up to 2·tpt new
//           tokens with the heads that share the K/V head (256 rows)
//   cost    of an item: the keys it sees, and PIECE for its start and end
//           (2.5 key tiles' time). Keys and not key tiles, because their sums
//           over items have a closed form without a division (counting tiles,
//           14 us passed until a CTA's item was found, now 4)
//   order   request by request, (chunk,) K/V head, item, key. The costs in this
//           order are cut into C equal shares, one a CTA, each end rounded down
//           to a key tile of its item: the lengths are on the device only, and
//           equal shares need no rule for uneven ones. An item that crosses
//           from one share to the next is finished by a merge of its parts.
//   chunk   a request with many items reads its keys once an item. CTAs with
//           equal shares stand at different keys of it, so what one reads has
//           left L2 before another needs it. Such a request's keys are
//           therefore cut into chunks of a share's length (or of what fits L2,
//           if that is more), and all items pass one chunk before any passes
//           the next: most shares are then one chunk of one item, and the CTAs
//           walk along the keys together. That pays while a context is not too
//           many shares long, for then an item has many parts: up to 4.5 where a
//           key and its value have 512 bytes (bf16, d = 128), else up to 2.5. Below
//           one share nothing is cut. 131072 keys, us with chunks and without,
//           half a second each (and shares a context):
//             bf16, d = 128  8 K/V heads, 16 items a head 1487 and 1720 (1.2), 10 993
//               and 1077 (1.9), 8 774 and 868 (2.4), 6 598 and 650 (3.2); 6 K/V heads,
//               7 532 and 575 (3.6), 6 470 and 496 (4.2); 4 heads, 10 506 and 499 (3.8),
//               9 463 and 493 (4.2), 8 427 and 407 (4.8); 2 heads, 16 422 and 385
//               (4.8), 6 223 and 162 (13)
//             bf16, d = 64, 8 heads  16 1123 and 1168 (1.2), 10 725 and 736 (1.9), 8 595
//               and 597 to 607 (2.4), 7 530 and 522 (2.7), 6 467 and 453 (3.2)
//             4-bit codes, d = 128, 8 heads  16 1842 and 1880 (1.2), 12 1401 and 1411
//               (1.6), 10 1186 and 1186 (1.9), 7 856 and 838 (2.7), 6 749 and 725 (3.2)
#pragma once

#include <cstdint>

#include "fa_common.h"
#include "fa_ptx.cuh"

#define FA_HD __host__ __device__ __forceinline__

namespace fa {
namespace ext {

constexpr int TK = 128;             // keys a tile
constexpr int PIECE = 320;          // an item's start and end, in keys (256: a prompt of 8192 tokens 1 us less, a mixed step 2 more; 384: 1 more each)
constexpr int MIN_SHARE = 5 * TK;  // a CTA's share is at least that: more than PIECE + TK, so that the ends of two
                                   // shares never round to one tile of an item
constexpr int MAX_CTAS = 152;
constexpr int CHUNK_ITEMS = 6;     // a request with fewer items a head is not cut into chunks,
constexpr int CHUNK_HALVES_512 = 9, CHUNK_HALVES = 5;  // nor one whose context is more half shares long
constexpr int MAX_PARTS = MAX_CTAS + (CHUNK_HALVES_512 + 1) / 2;  // of an item: one a share and one a chunk at most
static_assert(MIN_SHARE >= PIECE + 2 * TK, "");

typedef long long i64;

// One request: its first row of q, new tokens, cached tokens, items.
struct Request {
  int row0, n, len, items;
  FA_HD int base() const { return len - n; }  // position of its first new token
  // Behind the rows of the requests before it, which end at `floor` at most;
  // else taken for empty. Returns the floor of the next one. No row is worked
  // on twice then, and new tokens add up to T at most: the host's bounds on
  // parts and long items rest on that.
  FA_HD int behind(int floor) {
    if (n == 0) return floor;
    const int end = row0 + n;
    if (row0 < floor) n = items = 0;
    return max(floor, end);
  }
};

// Request b by its own two numbers; `broken` is set, and it is empty, if they
// are out of order or range. Where none is broken the starts do not decrease,
// so each is behind those before it.
FA_HD Request request_of(const Extend& p, int b, bool* broken) {
  Request r{0, 0, 0, 0};
  const int s = p.q_starts[b], e = p.q_starts[b + 1];
  const int len = p.seq_lens[b];
  if (s < 0 || e > p.T || e < s) {
    *broken = true;
    return r;
  }
  r.row0 = s, r.n = e - s;
  r.len = min(max(len, 0), p.max_blocks * p.bs);
  r.items = (r.n + 2 * p.tpt - 1) / (2 * p.tpt);
  return r;
}

// CHUNKS: of calls of which some request may be cut into chunks. (The code for
// it is left out of the others' kernels: they start from a cold instruction
// cache. 2777 tokens of 12 requests: 222 us with it, 209 without.)
template <bool CHUNKS>
struct Shape {
  int span;  // tokens an item: 2·tpt
  bool causal;
  int lc;    // keys a chunk, a multiple of TK
  int far;   // longer contexts are not cut into chunks

  // key tiles of `keys` (one at least, so that rows that see nothing are written)
  FA_HD static int tiles_of(int keys) { return max(1, (keys + TK - 1) / TK); }
  // keys item i sees: not decreasing in i
  FA_HD int keys(const Request& r, int i) const {
    return causal ? max(0, r.base() + min((i + 1) * span, r.n)) : r.len;
  }
  // Σ_{i' < i} keys(i')
  FA_HD i64 keys_before(const Request& r, int i) const {
    if (!causal) return static_cast<i64>(i) * r.len;
    const i64 full = min(i, r.items - 1);  // the last item may be shorter
    const i64 none = r.base() >= 0 ? 0 : min(static_cast<int>(full), -r.base() / span);
    const i64 s = (full - none) * r.base() + span * ((full * (full + 1) - none * (none + 1)) / 2);
    return i > full ? s + keys(r, r.items - 1) : s;
  }
  // the first item that sees more than x keys
  FA_HD int past(const Request& r, i64 x) const {
    if (r.len <= x) return r.items;
    if (!causal) return 0;
    const int d = static_cast<int>(x) - r.base();
    return d < 0 ? 0 : min(d / span, r.items - 1);
  }
  FA_HD bool chunked(const Request& r) const {
    return CHUNKS && r.items >= CHUNK_ITEMS && r.len > lc && r.len <= far;
  }
  FA_HD int chunks(const Request& r) const { return chunked(r) ? (r.len + lc - 1) / lc : 1; }
  // the first item that reaches chunk c
  FA_HD int reach(const Request& r, int c) const { return !CHUNKS || c == 0 ? 0 : past(r, static_cast<i64>(c) * lc); }
  // keys of item i in chunk c, which it reaches
  FA_HD int part(const Request& r, int c, int i) const {
    const int k = keys(r, i);
    return chunked(r) ? min(k - c * lc, lc) : k;
  }
  FA_HD int cost(const Request& r, int c, int i) const { return PIECE + part(r, c, i); }
  // Σ of the costs in chunk c of the items before i
  FA_HD i64 costs_before(const Request& r, int c, int i) const {
    if (!chunked(r)) return keys_before(r, i) + static_cast<i64>(i) * PIECE;
    const int i0 = reach(r, c), i1 = past(r, static_cast<i64>(c + 1) * lc);
    if (i <= i0) return 0;
    const int j = min(i, i1);  // from i1 on a whole chunk each
    return static_cast<i64>(i - i0) * PIECE + keys_before(r, j) - keys_before(r, i0) -
           static_cast<i64>(j - i0) * (static_cast<i64>(c) * lc) + static_cast<i64>(i - j) * lc;
  }
  // Σ_{1 <= c' < c} of the items that reach chunk c'
  FA_HD i64 reaches(const Request& r, int c) const {
    i64 s = 0;
    for (int x = 1; x < c; ++x) s += r.items - reach(r, x);
    return s;
  }
  // Σ of one head's costs in the chunks before c
  FA_HD i64 chunks_before(const Request& r, int c) const {
    if (c == 0) return 0;
    const int i = past(r, static_cast<i64>(c) * lc);
    return keys_before(r, i) + static_cast<i64>(r.items - i) * (static_cast<i64>(c) * lc) + (r.items + reaches(r, c)) * PIECE;
  }
  // a request's costs
  FA_HD i64 total(const Request& r, int heads) const {
    if (r.n == 0) return 0;
    return (chunked(r) ? chunks_before(r, chunks(r)) : costs_before(r, 0, r.items)) * heads;
  }
  // Items that pass more than one chunk are "long"; each of their chunks has a
  // part of its own: the first long item of chunk c, and one head's parts in
  // the chunks before c.
  FA_HD int first_long(const Request& r, int c) const { return past(r, static_cast<i64>(max(c, 1)) * lc); }
  FA_HD bool is_long(const Request& r, int i) const { return chunked(r) && keys(r, i) > lc; }
  FA_HD int long_before(const Request& r, int c) const {
    return c == 0 ? 0 : r.items - first_long(r, 0) + static_cast<int>(reaches(r, c));
  }
  // the tile at which a share's end x into an item's cost cuts it
  FA_HD static int tile_at(i64 x) { return x <= PIECE ? 0 : static_cast<int>((x - PIECE) / TK); }
};

// Sets the chunks' length: a share's, or what fits L2 if that is more. all: Σ of
// the keys that the items of all heads see.
FA_HD void set_chunks(Shape<true>* sh, const Extend& p, i64 all) {
  const i64 share = min((all / p.ctas + TK) / TK * TK, static_cast<i64>(1 << 29));
  sh->lc = max(static_cast<int>(share), p.lc);
  sh->far = static_cast<int>(min(share * p.chunk_halves / 2, static_cast<i64>(1 << 30)));
}

// The whole call's cut into `ctas` shares: share k is [start(k), start(k + 1)),
// the first `extra` one longer than the others.
struct Cut {
  i64 per;
  int ctas, extra;
  FA_HD Cut() : per(0), ctas(0), extra(0) {}
  FA_HD Cut(i64 cost, int most) {
    const i64 fit = cost / MIN_SHARE;
    ctas = fit < 1 ? 1 : fit > most ? most : static_cast<int>(fit);
    per = cost / ctas, extra = static_cast<int>(cost - per * ctas);
  }
  FA_HD i64 start(int k) const { return per * k + min(k, extra); }
  FA_HD int owner(i64 x) const {
    const i64 longer = (per + 1) * extra;
    return static_cast<int>(x < longer ? x / (per + 1) : extra + (x - longer) / per);
  }
};

// An item of one chunk, with what lies before it.
struct Place {
  Request r;
  int b;
  int floor;     // of the next request
  i64 request0;  // costs before the request
  int longs0;    // parts of long items before the request
  int c, hv, i;
  i64 item0;     // costs before the item
};

// Block-wide exclusive scan of one value a thread.
template <int NT>
__device__ __forceinline__ i64 block_scan(i64 v, i64* scratch, i64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  i64 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const i64 t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();  // the scratch may be in use
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  i64 below = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const i64 t = scratch[w];
    if (w < warp) below += t;
    all += t;
  }
  *total = all;
  return below + s - v;
}

// Block-wide exclusive maximum of one value a thread, none below 0.
template <int NT>
__device__ __forceinline__ int block_max(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s = max(s, t);
  }
  __syncthreads();  // the scratch may be in use
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  const int up = __shfl_up_sync(0xffffffffu, s, 1);
  int below = lane > 0 ? up : 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < NT / 32; ++w) {
    const int t = scratch[w];
    if (w < warp) below = max(below, t);
    all = max(all, t);
  }
  *total = all;
  return below;
}

struct PlanSmem {
  i64 scan[32];
  i64 request0, items0;
  Request r;
  int b, floor, longs0;
  int most[32];
};

// The call's requests, as a block goes through them: one a thread at a time.
template <int NT>
struct Requests {
  Request mine;     // this thread's of the first NT by its own numbers; all there are, mostly
  bool disordered;  // some request's are broken (reported)
  int floor;        // of the next tile
  int after;        // of the request after this thread's
  __device__ __forceinline__ Requests(const Extend& p, uint32_t* err) : mine{0, 0, 0, 0}, floor(0), after(0) {
    const int tid = static_cast<int>(threadIdx.x);
    bool broken = false;
    if (tid < p.B) mine = request_of(p, tid, &broken);
    for (int b = tid + NT; b < p.B; b += NT) request_of(p, b, &broken);
    if (broken) atomicExch(err, DEV_BAD_INDEX);
    disordered = __syncthreads_or(broken) != 0;
  }
  // Request b0 + threadIdx.x. By the whole block, tile after tile from b0 = 0.
  __device__ __forceinline__ Request tile(const Extend& p, int b0, PlanSmem* sm) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    bool broken;
    Request r = mine;
    if (b0 > 0) r = b < p.B ? request_of(p, b, &broken) : Request{0, 0, 0, 0};
    after = r.n > 0 ? r.row0 + r.n : 0;
    if (disordered) {
      if (b0 == 0) floor = 0;
      int all;
      const int before = block_max<NT>(after, sm->most, &all);
      after = r.behind(max(floor, before));
      floor = max(floor, all);
    }
    return r;
  }
};

// The call's cut, and the place of one of its items: with LONG = false of the
// one that share `want` begins in, with LONG = true of the want-th long item
// (its request and, in *items0, the long items before that). False: there is
// none. Run by a whole block; every thread knows the result, up to the request
// (locate has the rest). Sets sh->lc and far.
template <int NT, bool LONG, bool CHUNKS>
__device__ __forceinline__ bool plan(const Extend& p, Requests<NT>* rq, Shape<CHUNKS>* sh, PlanSmem* sm, int want, Cut* cut,
                                     Place* at, i64* items0) {
  const int tid = static_cast<int>(threadIdx.x);
  if constexpr (CHUNKS) {
    i64 k = 0, all;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
      const Request r = rq->tile(p, b0, sm);
      if (r.n > 0) k += sh->keys_before(r, r.items) * p.hv;
    }
    block_scan<NT>(k, sm->scan, &all);
    set_chunks(sh, p, all);
  }
  // costs before each thread's request; with more requests than threads, the total first
  i64 c = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) c += sh->total(rq->tile(p, b0, sm), p.hv);
  i64 total;
  const i64 before = block_scan<NT>(c, sm->scan, &total);
  *cut = Cut(total, p.ctas);
  if (tid == 0) sm->b = -1;
  const bool there = total > 0 && (LONG || want < cut->ctas);
  const i64 target = LONG || !there ? want : cut->start(want);
  i64 costs = 0, longs = 0, items = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const Request r = rq->tile(p, b0, sm);
    const i64 cost = p.B <= NT ? c : sh->total(r, p.hv);
    i64 sum = 0, sum_l = 0, sum_i = 0, l = 0, it = 0, e_l = 0, e_i = 0;
    const i64 e = p.B <= NT ? before : costs + block_scan<NT>(cost, sm->scan, &sum);
    if constexpr (CHUNKS) {
      if (r.n > 0 && sh->chunked(r)) {
        l = static_cast<i64>(sh->long_before(r, sh->chunks(r))) * p.hv;
        it = static_cast<i64>(r.items - sh->first_long(r, 0)) * p.hv;
      }
      e_l = longs + block_scan<NT>(l, sm->scan, &sum_l);
      e_i = items + block_scan<NT>(it, sm->scan, &sum_i);
    } else {
      __syncthreads();  // sm->b is set
    }
    const i64 key = LONG ? e_i : e, size = LONG ? it : cost;
    if (there && target >= key && target - key < size) {
      sm->b = b0 + tid, sm->r = r, sm->floor = rq->after;
      sm->request0 = e, sm->longs0 = static_cast<int>(e_l), sm->items0 = e_i;
    }
    costs += sum, longs += sum_l, items += sum_i;
  }
  __syncthreads();
  at->b = sm->b;
  if (at->b < 0) return false;
  at->r = sm->r;
  at->floor = sm->floor;
  at->request0 = sm->request0;
  at->longs0 = sm->longs0;
  *items0 = sm->items0;
  return true;
}

// The item that holds cost `x` of a request's; run by a whole warp.
template <bool CHUNKS>
__device__ __forceinline__ void locate(const Extend& p, const Shape<CHUNKS>& sh, i64 x, Place* at) {
  const int lane = threadIdx.x & 31;
  const Request& r = at->r;
  i64 rem = x - at->request0;
  int c = 0;
  if (sh.chunked(r)) {
    const int n_c = sh.chunks(r);
    for (int c0 = 0; c0 < n_c; c0 += 32) {
      const bool ok = c0 + lane < n_c && sh.chunks_before(r, c0 + lane) * p.hv <= rem;
      const int cnt = __popc(__ballot_sync(0xffffffffu, ok));
      if (cnt > 0) c = c0 + cnt - 1;
      if (cnt < 32) break;
    }
    rem -= sh.chunks_before(r, c) * p.hv;
  }
  at->c = c;
  at->hv = 0;
  // First the head, from one head's costs, then the item, by 32 probes at a
  // time; one copy of the code for both (it runs once, from a cold cache).
  int lo = sh.reach(r, c), hi = r.items;
  i64 found = 0;
  bool head = true;
#pragma unroll 1
  while (head || hi - lo > 1) {
    const int step = head ? 0 : (hi - lo + 31) / 32, probe = head ? hi : lo + lane * step;
    const i64 v = sh.costs_before(r, c, min(probe, hi));
    if (head) {
      for (int h0 = 0; h0 < p.hv; h0 += 32) {  // rem / v
        const int cnt = __popc(__ballot_sync(0xffffffffu, h0 + lane < p.hv && v * (h0 + lane) <= rem));
        if (cnt > 0) at->hv = h0 + cnt - 1;
        if (cnt < 32) break;
      }
      rem -= v * at->hv;
      head = false;
    } else {
      const int cnt = __popc(__ballot_sync(0xffffffffu, probe < hi && v <= rem));
      found = __shfl_sync(0xffffffffu, v, cnt - 1);
      lo += (cnt - 1) * step;
      hi = min(hi, lo + step);
    }
  }
  at->i = lo;
  at->item0 = x - (rem - found);  // found: the costs before item lo (0 if it is the first and only one)
}

// Where a piece's result goes: slots 2k and 2k + 1 are CTA k's first and last
// piece where its share cuts an item, the others hold whole chunks of long
// items; -1: the outputs themselves.
template <bool CHUNKS>
FA_HD int part_slot(const Extend& p, const Shape<CHUNKS>& sh, const Place& at, int k, bool start_cut, bool end_cut) {
  if (start_cut) return 2 * k;
  if (end_cut) return 2 * k + 1;
  if (!sh.is_long(at.r, at.i)) return -1;
  const int in_c = at.r.items - sh.first_long(at.r, at.c);
  return 2 * p.ctas + at.longs0 + p.hv * sh.long_before(at.r, at.c) + at.hv * in_c + at.i - sh.first_long(at.r, at.c);
}

// The parts that the shares make of one item of one chunk, in order: calls
// f(i, slot) for each; k: the share in which it begins. (An item cut once or
// more, and not a long one: slot 2k + 1 of the share k in which its first tile
// lies, then 2 (k + 1), 2 (k + 2) and so on.)
template <class F>
FA_HD int parts_of(const Extend& p, const Shape<true>& sh, const Cut& cut, const Place& at, int k, F f) {
  const int cost = sh.cost(at.r, at.c, at.i), tiles = Shape<true>::tiles_of(sh.part(at.r, at.c, at.i));
  const i64 end = at.item0 + cost;
  int n = 0;
  for (int lo = 0; lo < tiles; ++k) {
    const i64 e = cut.start(k + 1);
    const int hi = e >= end ? tiles : Shape<true>::tile_at(e - at.item0);
    if (hi <= lo) continue;
    f(n++, part_slot(p, sh, at, k, lo > 0, hi < tiles));
    lo = hi;
  }
  return n;
}

// What a CTA does of one item at a time.
struct Piece {
  int n, kt0;            // key tiles, the first of them; n = 0: no more pieces
  int b, kvh, head0, heads;
  int tok0, ntok;        // first row of q, tokens of the item
  int pos0, len;         // position of the first token; cached tokens
  int slot;              // -1: the outputs
  int n0, n1;            // key tiles that each query tile sees
  int unit0;             // the CTA's units before this piece
  int pad[2];
};
static_assert(sizeof(Piece) == 64, "");

// Share `cta`'s pieces in order, from the item it begins in: f(piece) for each,
// until that says false; false then. *entered: the item that the share begins
// within, if another share has its start (and it is not a long one).
template <bool CHUNKS, class F>
FA_HD bool walk(const Extend& p, const Shape<CHUNKS>& sh, const Cut& cut, int cta, Place at, ItemCut* entered, F f) {
  const i64 begin = cut.start(cta), end = cut.start(cta + 1);
  int lo = begin > at.item0 ? Shape<CHUNKS>::tile_at(begin - at.item0) : 0;
  const int G = p.H / p.Hkv, parts = p.hv / p.Hkv;
  Piece x{};  // n = 0
  while (true) {
    const Request& r = at.r;
    const int tiles = Shape<CHUNKS>::tiles_of(sh.part(r, at.c, at.i));
    const i64 item_end = at.item0 + sh.cost(r, at.c, at.i);
    const int hi = item_end <= end ? tiles : Shape<CHUNKS>::tile_at(end - at.item0);
    if (hi > lo) {
      x.unit0 += x.n;
      x.n = hi - lo;
      x.kt0 = (CHUNKS ? at.c * (sh.lc / TK) : 0) + lo;
      x.b = at.b;
      x.kvh = at.hv / parts;
      const int h0 = at.hv % parts * p.heads;
      x.head0 = x.kvh * G + h0;
      x.heads = min(p.heads, G - h0);
      const int t0 = at.i * sh.span;
      x.tok0 = r.row0 + t0;
      x.ntok = min(sh.span, r.n - t0);
      x.pos0 = r.base() + t0;
      x.len = r.len;
      x.slot = part_slot(p, sh, at, cta, lo > 0, hi < tiles);
      auto sees = [&](int g) {
        const int t = min((g + 1) * p.tpt, x.ntok);
        if (t <= g * p.tpt) return 0;
        const int keys = p.causal ? max(x.pos0 + t, 0) : x.len;
        return min(max((keys + TK - 1) / TK - x.kt0, 0), x.n);
      };
      x.n0 = sees(0), x.n1 = sees(1);
      if (!f(x)) return false;
      if (lo > 0 && !sh.is_long(r, at.i)) {  // the share's first piece at most
        int first = cut.owner(at.item0);
        if (Shape<CHUNKS>::tile_at(cut.start(first + 1) - at.item0) == 0) ++first;
        *entered = ItemCut{cut.owner(item_end - 1) - first + 1, cta - first, x.tok0, x.ntok, x.head0, x.heads};
      }
    }
    if (item_end >= end) return true;
    at.item0 = item_end;
    lo = 0;
    if (++at.i < r.items) continue;
    if (++at.hv == p.hv) {
      at.hv = 0;
      if (!CHUNKS || ++at.c == sh.chunks(r)) {
        if (sh.chunked(r)) at.longs0 += p.hv * sh.long_before(r, at.c);
        at.c = 0;
        do {  // costs are left, so there is a request with tokens
          bool broken;
          at.r = request_of(p, ++at.b, &broken);
          at.floor = at.r.behind(at.floor);
        } while (at.r.n == 0 && at.b + 1 < p.B);
      }
    }
    at.i = sh.reach(at.r, at.c);
  }
}

}  // namespace ext
}  // namespace fa
