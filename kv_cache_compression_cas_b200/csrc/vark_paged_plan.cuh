// How paged attention divides its work: the arithmetic of the plan, apart from
// the block-wide scan over the tables (vark_paged_attention.cu).  It compiles for
// the host as well, where the tests run it.
//
// Of the functions' parameter P: G (query heads a kv head), causal, by_group
// (/ G), by_heads (/ kv heads), tokens_per_tile (R / G), tile_step (weight from a
// row tile to the next under a causal mask), pg.heads (kv heads), pg.table_heads
// (rows of the length table a sequence has), entry<R, KT>(e) (row e of it).
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define VARK_PLAN __host__ __device__ __forceinline__
#else
#define VARK_PLAN inline
#endif

namespace vark {
namespace paged {

constexpr int kCtas = 148;             // one persistent CTA per SM
constexpr int kTileR = 256;            // rows of an item of the tiles kernel
constexpr int kTileKT = 128;           // keys of a key tile

template <typename T>
VARK_PLAN T lesser(T a, T b) { return b < a ? b : a; }
template <typename T>
VARK_PLAN T greater(T a, T b) { return a < b ? b : a; }

// Division by a number the host knows, by a product (a division costs 130
// cycles of latency, and several lie on the way to a CTA's first load).  Of
// the divisor d, with s = ceil(log2 d): mul = floor(2^32 (2^s - d) / d) + 1;
// x / d = (hi32(x mul) + x) >> s for 0 <= x < 2^31.
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv of(int d) {
    FastDiv f;
    f.shift = 0;
    while ((uint32_t(1) << f.shift) < uint32_t(d)) ++f.shift;
    f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - uint32_t(d))) / uint32_t(d) + 1);
    return f;
  }
  VARK_PLAN int operator()(int x) const {
#ifdef __CUDA_ARCH__
    const uint32_t hi = __umulhi(uint32_t(x), mul);
#else
    const uint32_t hi = uint32_t((uint64_t(uint32_t(x)) * mul) >> 32);
#endif
    return int((hi + uint32_t(x)) >> shift);
  }
};

// a / b of non-negative numbers, in 32 bits where they allow it (64 take ten
// times as long).
VARK_PLAN int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// An entry is one row of the length table: a sequence (shared pages, all kv
// heads) or a (sequence, head).  Its items, head after head and row tile after
// row tile, weigh what they cost, in sixteenths of a key: kItemCost tiles for
// starting and finishing one, and the keys its rows see -- which under a causal
// mask grow by the tokens of a tile from one row tile to the next, so the
// weights and their sums have a closed form.  (Equal weights left causal
// prompts with shares of 0.6 to 1.5 times the mean work.)
constexpr int kUnit = 16;
// Key tiles that an item counts for besides its own.  Of 0 / 1 / 2 / 3 / 5: 64
// sequences decoding 202 / 190 / 190 / 192 / 196 us, drafted tokens of 64
// channels 69 / 51 / 47 / 47 / 49, prompts 645 / 516 / 458 / 455 / 483.
constexpr int kItemCost = 2;
// Where there is a CTA for every item of 256 rows, cutting one up must save more
// than this many key tiles' time, which its partial results and the join cost:
// 200 tokens over 16 rows (32 heads of 128) 25.2 -> 19.4 us whole, 8 times 100
// over 1000 46.5 -> 35.9; at 9 one chunk of 64 over 700 loses 22.8 -> 25.1.
constexpr int kCutTiles = 6;
struct Entry {
  int first, n;            // first token, tokens
  int len;                 // cache rows
  int row_tiles, heads;    // row tiles of a head, kv heads of the entry
  int slope;               // weight of row tile t: weight0 + t * slope
  int64_t weight0;

  // Of `first`, `n` and `len`.
  template <int R, int KT, typename P>
  VARK_PLAN void weigh(const P& p) {
    row_tiles = (n * p.G + R - 1) / R;
    heads = p.pg.table_heads > 1 ? 1 : p.pg.heads;
    slope = p.causal && row_tiles > 1 ? p.tile_step : 0;
    const int seen0 = slope ? lesser(len, greater(0, len - n) + p.tokens_per_tile) : len;     // by the first row tile
    weight0 = int64_t(kUnit) * (int64_t(kItemCost) * KT + seen0);
  }
  VARK_PLAN int64_t sum(int t) const { return t * weight0 + int64_t(slope) * t * (t - 1) / 2; }   // of tiles 0 .. t-1
  VARK_PLAN int64_t head_units() const { return sum(row_tiles); }
  VARK_PLAN int64_t units() const { return heads * head_units(); }
  VARK_PLAN int64_t longest() const { return row_tiles == 0 ? 0 : weight0 + int64_t(row_tiles - 1) * slope; }
  VARK_PLAN void count_items() {                // every item weighs one unit
    slope = 0;
    weight0 = 1;
  }
  // The row tile that holds unit `off` of a head.
  VARK_PLAN int tile_of(int64_t off) const {
    int t;
    if (row_tiles == 1) return 0;
    if (slope == 0) {
      t = int(quotient(off, weight0));
    } else {
      const double lin = double(weight0) - 0.5 * slope;
      t = int((sqrt(lin * lin + 2.0 * slope * double(off)) - lin) / slope);
    }
    t = greater(0, lesser(row_tiles - 1, t));
    while (t > 0 && sum(t) > off) --t;
    while (t + 1 < row_tiles && sum(t + 1) <= off) ++t;
    return t;
  }
};

// Whether items that weigh `total`, the longest `tiles` key tiles, stay whole if
// there is a CTA for each.
template <int KT>
VARK_PLAN bool worth_whole(int tiles, int64_t total) {
  return (tiles - kCutTiles) * (int64_t(kUnit) * KT * kCtas) <= total;
}

// Where an item's key tiles lie in its units [from, to): after its fixed cost;
// the tile that unit u has come to (the last unit is the end of all tiles).
struct ItemPlace {
  int64_t from, to;
  int key_tiles;
  template <int KT>
  VARK_PLAN int tile_at(int64_t u) const {
    if (u >= to) return key_tiles;
    const int64_t k = (u - from) / (kUnit * KT) - kItemCost;
    return int(greater(int64_t(0), lesser(int64_t(key_tiles), k)));
  }
};

struct Share {
  int ctas;                // shares of the call: extra of them have per + 1 units, the others per
  int64_t per, extra;
  int64_t u0, u1;          // this CTA's units
  struct Place {
    int e;                 // an entry, its first unit, and itself
    int64_t base;
    Entry x;
  };
  Place first, last;       // where units u0 and u1 - 1 lie (last: on request)

  VARK_PLAN void split(int64_t total) {
    ctas = int(lesser(int64_t(kCtas), total));
    per = 1;
    extra = 0;
    if (total > kCtas) {
      per = quotient(total, kCtas);
      extra = total - per * kCtas;
    }
  }
  VARK_PLAN int64_t begin(int c) const { return per * c + lesser(int64_t(c), extra); }
  VARK_PLAN int holder(int64_t u) const {       // the share that unit u is in
    const int64_t wide = extra * (per + 1);
    return u < wide ? int(quotient(u, per + 1)) : int(extra + quotient(u - wide, per));
  }
};

// The runs of key tiles [k0, k1) of a share, item after item.
template <int R, int KT>
struct Segments {
  Entry x;
  int e, i;                // entry, head within it
  int64_t u, u1;           // next unit, end of the share
  ItemPlace at;            // the item of the segment
  int tile, h, k0, k1;

  template <typename P>
  VARK_PLAN void start(const P& p, const Share& s) {
    e = s.first.e;
    x = s.first.x;
    u = s.u0;
    u1 = s.u1;
    find(p, s.first.base, u);
  }
  template <typename P>
  VARK_PLAN bool next(const P& p) {
    while (u < u1) {
      if (u == at.to) step(p);
      const int64_t stop = lesser(at.to, u1);
      k0 = at.template tile_at<KT>(u);
      k1 = at.template tile_at<KT>(stop);
      u = stop;
      if (k0 < k1) return true;      // (else a share's end fell into the item's fixed cost)
    }
    return false;
  }
  VARK_PLAN bool whole() const { return k0 == 0 && k1 == at.key_tiles; }
  // The item of entry e, whose first unit is `base`, that holds unit v.
  template <typename P>
  VARK_PLAN void find(const P& p, int64_t base, int64_t v) {
    const int64_t per_head = x.head_units();
    int64_t off = v - base;
    i = x.heads == 1 ? 0 : int(quotient(off, per_head));
    off -= i * per_head;
    tile = x.tile_of(off);
    at.from = base + i * per_head + x.sum(tile);
    place(p);
  }
  template <typename P>
  VARK_PLAN void step(const P& p) {
    at.from = at.to;
    if (++tile == x.row_tiles) {
      tile = 0;
      if (++i == x.heads) {
        i = 0;
        const bool items = R == kTileR && x.weight0 == 1;      // (see count_items)
        do x = p.template entry<R, KT>(++e);
        while (x.row_tiles == 0);
        if (items) x.count_items();
      }
    }
    place(p);
  }
  template <typename P>
  VARK_PLAN void place(const P& p) {
    h = p.pg.table_heads > 1 ? e - p.by_heads(e) * p.pg.heads : i;
    at.to = at.from + x.weight0 + int64_t(tile) * x.slope;
    at.key_tiles = greater(1, (limit(p) + KT - 1) / KT);
  }
  // Keys that some row of the tile sees.
  template <typename P>
  VARK_PLAN int limit(const P& p) const {
    if (!p.causal) return x.len;
    const int last = lesser(x.n - 1, p.by_group(tile * R + R - 1));
    return greater(0, x.len - x.n + last + 1);
  }
};

// The item at one end of a share (0: its first unit's, 1: its last one's), if
// other shares may have parts of it; that of both ends counts as the first's.
template <int R, int KT, typename P>
VARK_PLAN bool cut_item(const P& p, const Share& s, int end, Segments<R, KT>& seg) {
  const Share::Place& at = end ? s.last : s.first;
  seg.e = at.e;
  seg.x = at.x;
  seg.find(p, at.base, end ? s.u1 - 1 : s.u0);
  if (seg.at.from >= s.u0 && seg.at.to <= s.u1) return false;             // all of it is here
  return end == 0 || s.u0 < seg.at.from;
}

// Share c's key tiles [k0, k1) of an item, and the place of its partial result: of
// the two a CTA has, the first for an item begun before its share.
template <int KT>
VARK_PLAN void part_of(const ItemPlace& item, const Share& s, int c, int& k0, int& k1) {
  k0 = item.template tile_at<KT>(greater(item.from, s.begin(c)));
  k1 = item.template tile_at<KT>(lesser(item.to, s.begin(c + 1)));
}
VARK_PLAN int part_slot(int c, int k0) { return 2 * c + (k0 == 0 ? 1 : 0); }

}  // namespace paged
}  // namespace vark
