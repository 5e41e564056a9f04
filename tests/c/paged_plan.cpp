// The plan of paged attention (csrc/vark_paged_plan.cuh) for the host: the shares,
// segments and joins of a call, over lengths given as arrays.  The scan over the
// tables, which the device does block-wide, is a loop here.
#include "vark_paged_plan.cuh"

using namespace vark::paged;

namespace {

struct Call {
  int G, causal, tokens_per_tile, tile_step;
  FastDiv by_group, by_heads;
  struct { int heads, table_heads; } pg;
  int entries;
  const int *n, *len;        // of a sequence; of an entry

  template <int R, int KT>
  Entry entry(int e) const {
    Entry x;
    x.first = 0;
    x.n = n[pg.table_heads > 1 ? by_heads(e) : e];
    x.len = len[e];
    x.weigh<R, KT>(*this);
    return x;
  }
};

struct Out {
  int* to;
  int rows, most;
  void put(int a, int b, int c, int d, int e, int f, int g, int h) {
    if (rows < most) {
      int* r = to + 8 * rows;
      r[0] = a; r[1] = b; r[2] = c; r[3] = d; r[4] = e; r[5] = f; r[6] = g; r[7] = h;
    }
    ++rows;
  }
};

template <int R>
Share::Place locate(const Call& p, int64_t unit, bool one_each) {
  int64_t base = 0;
  for (int e = 0; e < p.entries; ++e) {
    Entry x = p.entry<R, kTileKT>(e);
    if (one_each) x.count_items();
    if (unit < base + x.units()) return Share::Place{e, base, x};
    base += x.units();
  }
  return Share::Place{-1, base, Entry{}};
}

template <int R>
int run(const Call& p, int* segments, int n_segments, int* joins, int n_joins, int64_t* info) {
  int64_t total = 0, items = 0, longest = 0;
  for (int e = 0; e < p.entries; ++e) {
    const Entry x = p.entry<R, kTileKT>(e);
    total += x.units();
    items += int64_t(x.heads) * x.row_tiles;
    longest = greater(longest, x.longest());
  }
  const int64_t tile = int64_t(kUnit) * kTileKT;
  const bool one_each =
      R == kTileR && worth_whole<kTileKT>(int((longest + tile - 1) / tile), total) && items <= kCtas;
  if (one_each) total = items;
  Share s;
  s.split(total);
  Out seg_out{segments, 0, n_segments}, join_out{joins, 0, n_joins};
  for (int c = 0; c < s.ctas; ++c) {
    s.u0 = s.begin(c);
    s.u1 = s.begin(c + 1);
    s.first = locate<R>(p, s.u0, one_each);
    s.last = locate<R>(p, s.u1 - 1, one_each);
    if (s.first.e < 0 || s.last.e < 0 || s.holder(s.u0) != c || s.holder(s.u1 - 1) != c) return -1;
    Segments<R, kTileKT> g;
    g.start(p, s);
    while (g.next(p)) seg_out.put(c, g.e, g.h, g.tile, g.k0, g.k1, g.at.key_tiles, g.limit(p));
    for (int end = 0; end < 2; ++end) {
      Segments<R, kTileKT> at;
      if (!cut_item(p, s, end, at)) continue;
      const int c0 = s.holder(at.at.from), c1 = s.holder(at.at.to - 1);
      for (int q = c0; q <= c1; ++q) {
        int k0, k1;
        part_of<kTileKT>(at.at, s, q, k0, k1);
        join_out.put(c, at.e, at.h, at.tile, q, k0, k1, k0 < k1 ? part_slot(q, k0) : -1);
      }
    }
  }
  info[0] = total;
  info[1] = one_each;
  info[2] = s.ctas;
  info[3] = seg_out.rows;
  info[4] = join_out.rows;
  return 0;
}

}  // namespace

extern "C" {

int constant(int which) {
  const int c[] = {kCtas, kTileR, kTileKT, kUnit, kItemCost, kCutTiles};
  return c[which];
}
int fast_div(int x, int d) { return FastDiv::of(d)(x); }
int64_t divide(int64_t a, int64_t b) { return quotient(a, b); }
// The row tile of unit `off`, and the units before tile t.
int tile_of(int row_tiles, int slope, int64_t weight0, int64_t off) {
  Entry x{};
  x.row_tiles = row_tiles;
  x.slope = slope;
  x.weight0 = weight0;
  return x.tile_of(off);
}
int64_t tile_sum(int slope, int64_t weight0, int t) {
  Entry x{};
  x.slope = slope;
  x.weight0 = weight0;
  return x.sum(t);
}
// n [B]; len [B], or [B][heads] with head_pages.  A row of `segments`: cta, entry,
// head, row tile, k0, k1, key tiles of the item, keys it sees; of `joins`: cta,
// entry, head, row tile, share, k0, k1, slot (-1: no part).
int plan(int R, int B, const int* n, const int* len, int heads, int head_pages, int G, int causal, int* segments,
         int n_segments, int* joins, int n_joins, int64_t* info) {
  Call p;
  p.G = G;
  p.causal = causal;
  p.tokens_per_tile = R / G;
  p.tile_step = R * kUnit / G;
  p.by_group = FastDiv::of(G);
  p.by_heads = FastDiv::of(heads);
  p.pg.heads = heads;
  p.pg.table_heads = head_pages ? heads : 1;
  p.entries = B * p.pg.table_heads;
  p.n = n;
  p.len = len;
  if (R == 16) return run<16>(p, segments, n_segments, joins, n_joins, info);
  if (R == 32) return run<32>(p, segments, n_segments, joins, n_joins, info);
  return run<kTileR>(p, segments, n_segments, joins, n_joins, info);
}
}
