// The cut of a chunk call (fa_extend_plan.cuh), evaluated on the host and
// compared with an enumeration: tests/test_extend_plan.py builds and calls it.
#include <algorithm>
#include <map>
#include <set>
#include <tuple>
#include <vector>

#include "fa_extend_plan.cuh"

#pragma nv_diag_suppress 20013, 20015  // host lambdas, called on the host only

using namespace fa;
using namespace fa::ext;

#define CHECK(x) \
  do {           \
    if (!(x)) return __LINE__; \
  } while (0)

namespace {

struct Item {  // of one chunk
  int b, c, hv, i, tiles;
  i64 item0, request0;
  int longs0, cost;
};

}  // namespace

// Chunks of the longest cut request (1: none is cut), long items, the largest
// slot, requests taken for empty, keys a chunk.
template <bool CHUNKS>
static int check(const Extend& p, int halves, int* out) {
  const int T = p.T, B = p.B, G = p.H / p.Hkv, span = 2 * p.tpt, parts = p.hv / p.Hkv, bs = p.bs, max_blocks = p.max_blocks;
  const int *starts = p.q_starts, *lens = p.seq_lens;
  const bool causal = p.causal;
  CHECK(p.ctas >= 1 && p.ctas <= MAX_CTAS && p.heads * parts >= G && p.tpt * p.heads <= 128);

  // Which requests there are, from the rule as it is documented.
  std::vector<Request> rq(B);
  int dropped = 0, floor = 0;
  i64 tokens = 0;
  for (int b = 0; b < B; ++b) {
    const int s = starts[b], e = starts[b + 1];
    auto ordered = [&](int x) { return starts[x] >= 0 && starts[x + 1] <= T && starts[x + 1] >= starts[x]; };
    bool there = ordered(b) && e > s;
    for (int x = 0; x < b; ++x) there = there && !(ordered(x) && starts[x + 1] > starts[x] && starts[x + 1] > s);
    bool broken = false;
    rq[b] = request_of(p, b, &broken);
    CHECK(broken == !ordered(b));
    floor = rq[b].behind(floor);
    CHECK(rq[b].n == (there ? e - s : 0));
    if (!there && (broken || e > s)) ++dropped;
    if (there) {
      CHECK(rq[b].row0 == s && rq[b].items == (e - s + span - 1) / span);
      CHECK(rq[b].len == std::min<i64>(std::max(lens[b], 0), static_cast<i64>(max_blocks) * bs));
      tokens += e - s;
    }
  }
  CHECK(tokens <= T);

  // Every item of every chunk, in order, its costs one by one.
  auto keys_of = [&](const Request& r, int i) {
    i64 most = 0;
    for (int t = i * span; t < std::min((i + 1) * span, r.n); ++t)
      most = std::max<i64>(most, causal ? std::max(r.len - r.n + t + 1, 0) : r.len);
    return static_cast<int>(most);
  };
  Shape<CHUNKS> sh{span, p.causal, p.lc, 0};
  std::vector<std::vector<int>> keys(B);
  i64 all = 0;
  for (int b = 0; b < B; ++b) {
    i64 sum = 0;
    for (int i = 0; i < rq[b].items; ++i) {
      keys[b].push_back(keys_of(rq[b], i));
      CHECK(sh.keys(rq[b], i) == keys[b][i] && sh.keys_before(rq[b], i) == sum);
      sum += keys[b][i];
    }
    if (rq[b].n > 0) CHECK(sh.keys_before(rq[b], rq[b].items) == sum);
    all += sum * p.hv;
  }
  if constexpr (CHUNKS) set_chunks(&sh, p, all);
  CHECK(!CHUNKS || sh.lc == std::max<i64>(p.lc, (all / p.ctas + TK) / TK * TK));
  CHECK(sh.lc % TK == 0 && sh.lc > 0);
  std::vector<Item> items;
  std::map<std::tuple<int, int, int>, int> tiles_left;  // (request, head, item): tiles not yet dealt out
  i64 total = 0;
  int longs0 = 0, n_long = 0, most_chunks = 1;
  for (int b = 0; b < B; ++b) {
    const Request& r = rq[b];
    if (r.n == 0) continue;
    const bool cut = CHUNKS && r.items >= 6 && r.len > sh.lc && 2ll * r.len <= halves * ((all / p.ctas + TK) / TK * TK);
    CHECK(sh.chunked(r) == cut);
    const int chunks = cut ? (r.len + sh.lc - 1) / sh.lc : 1;
    CHECK(sh.chunks(r) == chunks);
    most_chunks = std::max(most_chunks, chunks);
    const i64 request0 = total;
    int long_parts = 0;
    for (int c = 0; c < chunks; ++c) {
      i64 row = 0;
      if (c > 0 || cut) CHECK(sh.chunks_before(r, c) * p.hv == total - request0);
      if (cut) CHECK(sh.long_before(r, c) == long_parts);
      for (int hv = 0; hv < p.hv; ++hv) {
        row = 0;
        bool first = true;
        for (int i = 0; i < r.items; ++i) {
          if (c > 0 && keys[b][i] <= c * sh.lc) continue;
          if (first) CHECK(sh.reach(r, c) == i);
          first = false;
          const int mine = cut ? std::min(keys[b][i] - c * sh.lc, sh.lc) : keys[b][i];
          const int n = std::max(1, (mine + TK - 1) / TK);
          CHECK(sh.cost(r, c, i) == PIECE + mine && sh.costs_before(r, c, i) == row);
          items.push_back(Item{b, c, hv, i, n, total, request0, longs0, PIECE + mine});
          tiles_left[{b, hv, i}] += n;
          row += PIECE + mine, total += PIECE + mine;
          const bool is_long = cut && keys[b][i] > sh.lc;
          CHECK(sh.is_long(r, i) == is_long);
          if (hv == 0 && is_long) ++long_parts;
          if (c == 0 && is_long) ++n_long;
        }
        CHECK(sh.costs_before(r, c, r.items) == row);
      }
    }
    CHECK(sh.total(r, p.hv) == total - request0);
    longs0 += long_parts * p.hv;
  }
  for (const auto& t : tiles_left)
    CHECK(t.second == std::max(1, (keys[std::get<0>(t.first)][std::get<2>(t.first)] + TK - 1) / TK));
  CHECK(n_long <= p.n_long && 2 * p.ctas + longs0 <= p.n_slots);
  out[0] = most_chunks, out[1] = n_long, out[2] = -1, out[3] = dropped, out[4] = sh.lc;
  if (total == 0) return 0;

  // The shares' pieces: every tile once, every slot once.
  const Cut cut(total, p.ctas);
  CHECK(cut.start(0) == 0 && cut.start(cut.ctas) == total && cut.ctas <= p.ctas);
  std::set<int> slots;
  std::map<std::tuple<int, int, int>, std::map<int, Piece>> dealt;  // by first tile
  std::vector<ItemCut> cuts(p.ctas, ItemCut{});
  std::vector<Place> places(cut.ctas);
  size_t at_item = 0;
  for (int k = 0; k < cut.ctas; ++k) {
    const i64 begin = cut.start(k);
    CHECK(cut.owner(begin) == k && cut.owner(cut.start(k + 1) - 1) == k);
    while (items[at_item].item0 + items[at_item].cost <= begin) ++at_item;
    const Item& x = items[at_item];
    Place at{rq[x.b], x.b, 0, x.request0, x.longs0, x.c, x.hv, x.i, x.item0};
    for (int b = 0, f = 0; b <= x.b; ++b) {
      bool broken;
      Request r = request_of(p, b, &broken);
      at.floor = f = r.behind(f);
    }
    int line = 0, units = 0;
    auto take = [&](const Piece& y) -> int {
      const int hv = y.kvh * parts + (y.head0 - y.kvh * G) / p.heads;
      const Request& r = rq[y.b];
      CHECK(y.n > 0 && r.n > 0 && hv < p.hv && (y.tok0 - r.row0) % span == 0 && y.len == r.len);
      const int i = (y.tok0 - r.row0) / span;
      CHECK(i < r.items && y.ntok == std::min(span, r.n - i * span) && y.pos0 == r.len - r.n + i * span);
      CHECK(y.head0 >= y.kvh * G && y.heads == std::min(p.heads, (y.kvh + 1) * G - y.head0) && y.heads > 0);
      CHECK(y.unit0 == units);
      units += y.n;
      for (int g = 0; g < 2; ++g) {
        int most = 0;
        for (int t = g * p.tpt; t < std::min((g + 1) * p.tpt, y.ntok); ++t)
          most = std::max(most, causal ? y.pos0 + t + 1 : y.len);
        CHECK((g ? y.n1 : y.n0) == std::min(std::max((most + TK - 1) / TK - y.kt0, 0), y.n));
      }
      CHECK(y.slot >= -1 && y.slot < p.n_slots);
      if (y.slot >= 0) CHECK(slots.insert(y.slot).second);
      CHECK(dealt[std::make_tuple(y.b, hv, i)].emplace(y.kt0, y).second);
      return 0;
    };
    CHECK(walk(p, sh, cut, k, at, &cuts[k], [&](const Piece& y) { return (line = take(y)) == 0; }) || line != 0);
    if (line) return line;
    places[k] = at;
  }
  for (const auto& t : tiles_left) {
    const auto it = dealt.find(t.first);
    CHECK(it != dealt.end());
    int next = 0;
    for (const auto& y : it->second) {
      CHECK(y.first == next);
      next += y.second.n;
    }
    CHECK(next == t.second);
    CHECK((it->second.size() == 1) == (it->second.begin()->second.slot == -1));
  }
  CHECK(dealt.size() == tiles_left.size());
  out[2] = slots.empty() ? -1 : *slots.rbegin();

  // What the merge joins: cut items as their CTAs noted them, then the long ones.
  std::map<std::tuple<int, int, int>, int> joined;
  std::set<std::tuple<int, int>> noted;
  CHECK(cuts[0].parts == 0);
  for (int k = 1; k < p.ctas; ++k) {
    const ItemCut& c = cuts[k];
    if (c.parts == 0) continue;
    CHECK(k < cut.ctas && c.nth >= 1 && c.nth < c.parts && c.parts <= MAX_PARTS);
    const int first = k - c.nth;
    CHECK(first >= 0 && noted.insert({first, c.nth}).second);
    const int kvh = c.head0 / G, hv = kvh * parts + (c.head0 - kvh * G) / p.heads;
    int b = 0;
    while (!(rq[b].n > 0 && c.tok0 >= rq[b].row0 && c.tok0 < rq[b].row0 + rq[b].n)) ++b;
    const int i = (c.tok0 - rq[b].row0) / span;
    CHECK(!sh.is_long(rq[b], i));
    const auto& pieces = dealt[std::make_tuple(b, hv, i)];
    CHECK(static_cast<int>(pieces.size()) == c.parts);
    int n = 0;
    for (const auto& y : pieces) {
      CHECK(y.second.slot == (n == 0 ? 2 * first + 1 : 2 * (first + n)));
      CHECK(y.second.tok0 == c.tok0 && y.second.ntok == c.ntok && y.second.head0 == c.head0 && y.second.heads == c.heads);
      ++n;
    }
    ++joined[std::make_tuple(b, hv, i)];
  }
  int order = 0;
  for (const Item& x : items) {
    const Request& r = rq[x.b];
    const auto key = std::make_tuple(x.b, x.hv, x.i);
    if (!sh.is_long(r, x.i)) {
      const int pieces = static_cast<int>(dealt[key].size());
      CHECK(joined[key] == pieces - 1);
      continue;
    }
    if (x.c > 0) continue;
    ++order;
    if constexpr (CHUNKS) {
      std::vector<int> got;
      const int n_c = (keys[x.b][x.i] + sh.lc - 1) / sh.lc;
      for (int c = 0; c < n_c; ++c) {
        Place at{r, x.b, 0, x.request0, x.longs0, c, x.hv, x.i, 0};
        at.item0 = x.request0 + sh.chunks_before(r, c) * p.hv + sh.costs_before(r, c, r.items) * x.hv + sh.costs_before(r, c, x.i);
        parts_of(p, sh, cut, at, cut.owner(at.item0), [&](int, int slot) { got.push_back(slot); });
      }
      CHECK(got.size() <= static_cast<size_t>(MAX_PARTS) && got.size() == dealt[key].size());
      size_t n = 0;
      for (const auto& y : dealt[key]) CHECK(got[n++] == y.second.slot);
    }
  }
  CHECK(order == n_long);
  return 0;
}

// 0, or the line of the check that failed.
extern "C" int plan_check(int T, int B, int H, int Hkv, int d, int bs, int max_blocks, int causal, int q4,
                          const int* starts, const int* lens, int* out) {
  Extend p{};
  p.T = T, p.B = B, p.H = H, p.Hkv = Hkv, p.bs = bs, p.max_blocks = max_blocks, p.causal = causal != 0;
  p.q_starts = starts, p.seq_lens = lens;
  extend_sizes(&p, d, q4 != 0);
  const int halves = d == 128 && !q4 ? 9 : 5;
  return p.may_chunk ? check<true>(p, halves, out) : check<false>(p, halves, out);
}
