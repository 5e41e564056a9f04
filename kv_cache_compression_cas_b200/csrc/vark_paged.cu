// Row operators of the serving path:
//   * vark_qk_norm_rope: norm of every query and key row and the position
//     rotation, one pass;
//   * vark_paged_append: the same on the keys of a chunk, written with the
//     values to their rows of a paged cache.
//
// Mathematics (row x of D channels, fp32): RMS y = x / sqrt(sum(x^2) / D + eps)
// * w, L2 y = x / max(sqrt(sum(x^2)), eps) * w; a pair (a, b) of the rotated
// channels becomes (a cos - b sin, a sin + b cos).  One rounding, at the store.
//
// Layout: D / 16 lanes hold a row, two vectors of 8 channels each.  The two are
// the halves of the lane's 8 rotated pairs (half-split pairs are R / 2 apart),
// so the rotation needs no exchange between lanes and the sum of squares
// log2(D / 16) shuffles.  A warp takes one token and up to 16 heads of it: all
// rows are loaded first, and the token's cosines and sines are read once for
// all of them.
#include <cfloat>

#include "vark_paged.cuh"

namespace vark {
namespace paged {

// Both kernels are bound by HBM at large sizes, by one chain of dependent loads
// (position -> cosines) at small ones and, in between, by the latency of the rows'
// loads, too few of which are in flight (8 ragged chunks of 79 MB: 17 us, DRAM at
// 28%): the position is asked for before
// the rows, rows are read and written as streams, and blocks are small so that
// a finished one makes room at once.  Measured on the last scale of a batch of
// 8 (32768 tokens of 16 + 16 heads of 128): 92 to 98 us, 5.5 to 5.8 TB/s; 128-thread blocks
// 100, the position after the rows 111 with plain stores, 8 heads a warp 105.
constexpr int kRowThreads = 64;

struct Rotation {
  const float* table;       // [rope_len][2][dim / 2], or null
  const int32_t* positions; // [tokens]
  int len, dim, pairs;
};

// A lane's two vectors of a row (v: their indices) and what turns them.
template <int D>
struct Lane {
  int v[2];
  bool turns;              // else both pass through
  float c[8], s[8];        // of pair e; adjacent pairs: 0-3 of the first vector, 4-7 of the second

  VARK_DEV void place(const Rotation& r, int li) {
    const int half = r.table != nullptr ? r.dim >> 4 : 0;      // vectors in half the rotated channels
    turns = li < half;
    v[0] = turns ? li : 2 * li;
    v[1] = turns ? li + half : 2 * li + 1;
  }
  VARK_DEV void load(const Rotation& r, int pos) {
    if (!turns) return;
    const float* row = r.table + int64_t(pos) * r.dim;
    const int half = r.dim >> 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = r.pairs ? v[e] * 4 : v[0] * 8 + e * 4;
      const float4 cc = *reinterpret_cast<const float4*>(row + j);
      const float4 ss = *reinterpret_cast<const float4*>(row + half + j);
      c[4 * e] = cc.x; c[4 * e + 1] = cc.y; c[4 * e + 2] = cc.z; c[4 * e + 3] = cc.w;
      s[4 * e] = ss.x; s[4 * e + 1] = ss.y; s[4 * e + 2] = ss.z; s[4 * e + 3] = ss.w;
    }
  }
};

template <int DT>
VARK_DEV void unpack8(const uint4& w, float* x) {
  unpack2<DT>(w.x, x[0], x[1]);
  unpack2<DT>(w.y, x[2], x[3]);
  unpack2<DT>(w.z, x[4], x[5]);
  unpack2<DT>(w.w, x[6], x[7]);
}
template <int DT>
VARK_DEV uint4 pack8(const float* x) {
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
}

// Norm and rotation of one row, in place (every lane of the warp calls it;
// lanes without a row pass zeros).
template <int DT, int D>
VARK_DEV void norm_rotate(uint4 (&w)[2], int norm, float eps, bool weighted, const float (&wt)[16], const Rotation& rot,
                          const Lane<D>& ln) {
  float x[16];
  unpack8<DT>(w[0], x);
  unpack8<DT>(w[1], x + 8);
  if (norm != VARK_NORM_NONE) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s0 = fmaf(x[e], x[e], s0);
      s1 = fmaf(x[8 + e], x[8 + e], s1);
    }
    float ss = s0 + s1;
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float len = sqrtf(ss);                   // (a NaN stays one: fmaxf would give eps for it)
    const float inv = norm == VARK_NORM_RMS ? 1.f / sqrtf(ss * (1.f / D) + eps) : 1.f / (len < eps ? eps : len);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= inv;
  }
  if (weighted) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= wt[e];
  }
  if (ln.turns) {
    if (rot.pairs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * ln.c[e] - b * ln.s[e];
        x[2 * e + 1] = a * ln.s[e] + b * ln.c[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[e], b = x[8 + e];
        x[e] = a * ln.c[e] - b * ln.s[e];
        x[8 + e] = a * ln.s[e] + b * ln.c[e];
      }
    }
  }
  w[0] = pack8<DT>(x);
  w[1] = pack8<DT>(x + 8);
}

// -1: the token is padding (not written); -2: position outside the table.
VARK_DEV int token_position(const Rotation& r, int64_t token) {
  if (r.table == nullptr) return 0;
  const int p = r.positions[token];
  return p < 0 ? -1 : (p >= r.len ? -2 : p);
}

VARK_DEV void load_weight(const float* w, const int (&v)[2], float (&wt)[16]) {
  if (w == nullptr) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 a = *reinterpret_cast<const float4*>(w + v[e >> 1] * 8 + (e & 1) * 4);
    wt[4 * e] = a.x; wt[4 * e + 1] = a.y; wt[4 * e + 2] = a.z; wt[4 * e + 3] = a.w;
  }
}

struct RowTensor {
  const uint16_t* src;
  uint16_t* dst;
  const float* weight;
  int64_t ss[3], ds[3];    // batch, token, head strides (elements)
  int heads;
};

struct NormRopeParams {
  RowTensor t[2];          // queries, keys
  int T, tokens;           // tokens = B * T
  int q_blocks;            // grid rows of the queries' heads; the keys' follow
  int norm;
  float eps;
  Rotation rot;
  int32_t* status;
};

constexpr int kQkHeads = 16;       // heads of a warp's token

// Blocks an SM, that is registers: 128 channels 10 blocks of 96 (above: 92 us;
// 12 of 80 spill: 100), 64 channels, which hold half as many rows, 14 of 72
// (8191 tokens of 32 + 8 heads out of a fused projection: 20.4 us, 4.1 TB/s;
// 12 of 80 21.5, 10 of 95 24.3).
template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads, D == 64 ? 14 : 10)
norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kIters = kQkHeads / kRows;
  const int lane = threadIdx.x & 31, li = lane % kLanes;
  const int token = int(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  grid_release();
  grid_wait();
  if (token >= p.tokens) return;
  const bool keys = int(blockIdx.y) >= p.q_blocks;
  const RowTensor& t = p.t[keys];
  const int h0 = (int(blockIdx.y) - (keys ? p.q_blocks : 0)) * kQkHeads + lane / kLanes;
  const int b = token / p.T, i = token - b * p.T;
  const uint16_t* src = t.src + b * t.ss[0] + i * t.ss[1];
  uint16_t* dst = t.dst + b * t.ds[0] + i * t.ds[1];
  Lane<D> ln;
  ln.place(p.rot, li);
  const int pos = token_position(p.rot, token);
  uint4 w[kIters][2];
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    w[r][0] = w[r][1] = make_uint4(0u, 0u, 0u, 0u);
    if (h < t.heads) {
      w[r][0] = ld_stream(src + h * t.ss[2] + ln.v[0] * 8);
      w[r][1] = ld_stream(src + h * t.ss[2] + ln.v[1] * 8);
    }
  }
  if (pos < 0) {
    if (pos == -2 && lane == 0) record(p.status, VARK_E_SHAPE);
    return;
  }
  ln.load(p.rot, pos);
  float wt[16];
  load_weight(t.weight, ln.v, wt);
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    norm_rotate<DT, D>(w[r], p.norm, p.eps, t.weight != nullptr, wt, p.rot, ln);
    if (h < t.heads) {
      __stcs(reinterpret_cast<uint4*>(dst + h * t.ds[2] + ln.v[0] * 8), w[r][0]);
      __stcs(reinterpret_cast<uint4*>(dst + h * t.ds[2] + ln.v[1] * 8), w[r][1]);
    }
  }
}

struct AppendParams {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ks[2], vs[2];    // token, head strides (elements)
  uint16_t* k_pages;
  uint16_t* v_pages;
  Pages pg;
  const int32_t* cu;       // [B + 1]
  int B, tokens;
  const float* weight;
  int norm;
  float eps;
  Rotation rot;
  int32_t* status;
};

// The last sequence b with cu[b] <= token (32-way search by the warp): the one
// that holds the token if any does.  -1: before the first sequence.
VARK_DEV int find_sequence(const int32_t* cu, int B, int64_t token, int lane) {
  int lo = 0, n = B + 1;        // the answer is lo + (something below n) - or before lo
  for (;;) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && cu[lo + min(at, n - 1)] <= token);
    if (m == 0) return lo - 1;   // only on the first round: later ones start at a hit
    const int last = 31 - __clz(m);
    lo += last * step;
    if (step == 1) return lo;
    n = min(step, n - last * step);
  }
}

constexpr int kKvHeads = 8;        // heads of a warp's token

// 12 blocks an SM (80 registers): 46 to 48.6 us for 4 x 4096 tokens of 16 heads
// into head pages (5.5 to 5.8 TB/s); unbounded (91 registers) 47.5, 4 heads a warp 50.  L2
// prefetches ahead of the wait: 51 (ragged chunks of 79 MB 15.6 instead of 16.5).
template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads, 12) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kIters = (kKvHeads + kRows - 1) / kRows;
  const int lane = threadIdx.x & 31, li = lane % kLanes;
  const int token = int(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  grid_release();
  grid_wait();
  if (token >= p.tokens) return;
  const int h0 = int(blockIdx.y) * kKvHeads + lane / kLanes;
  Lane<D> ln;
  ln.place(p.rot, li);
  // The position first, and the rows before the search: each starts a chain
  // of dependent loads.
  const int pos = token_position(p.rot, token);
  const uint16_t* ks = p.k + token * p.ks[0];
  const uint16_t* vs = p.v + token * p.vs[0];
  uint4 kw[kIters][2], vw[kIters][2];
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    kw[r][0] = kw[r][1] = vw[r][0] = vw[r][1] = make_uint4(0u, 0u, 0u, 0u);
    if (h < p.pg.heads) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kw[r][e] = ld_stream(ks + h * p.ks[1] + ln.v[e] * 8);
        vw[r][e] = ld_stream(vs + h * p.vs[1] + ln.v[e] * 8);
      }
    }
  }
  const int b = find_sequence(p.cu, p.B, token, lane);
  // Offsets that descend or leave the chunk are recorded, 32 a warp.
  if (blockIdx.y == 0) {
    for (int64_t e = int64_t(token) * 32 + lane; e < p.B; e += int64_t(p.tokens) * 32) {
      const int lo = p.cu[e], hi = p.cu[e + 1];
      if (lo < 0 || hi < lo || hi > p.tokens) record(p.status, VARK_E_SHAPE);
    }
  }
  if (b < 0 || b >= p.B || pos == -1) return;   // outside every sequence, or padding
  if (pos == -2) {
    if (lane == 0) record(p.status, VARK_E_SHAPE);
    return;
  }
  const int first = p.cu[b], end = p.cu[b + 1];
  if (first < 0 || end > p.tokens || token >= end) return;      // offsets outside the chunk, or descending
  const int n = end - first;
  ln.load(p.rot, pos);
  float wt[16];
  load_weight(p.weight, ln.v, wt);
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    norm_rotate<DT, D>(kw[r], p.norm, p.eps, p.weight != nullptr, wt, p.rot, ln);
    if (h >= p.pg.heads) continue;
    const int64_t e = int64_t(b) * p.pg.table_heads + (p.pg.table_heads > 1 ? h : 0);
    const int len = p.pg.len[e];
    const bool fits = len >= 0 && (len - 1) >> p.pg.log2_page < p.pg.max_pages;
    const int row = len - n + (token - first);
    if (fits && row < 0) continue;              // the cache holds only the chunk's last len rows
    const int64_t page = fits ? p.pg.table[e * p.pg.max_pages + (row >> p.pg.log2_page)] : -1;
    if (page < 0 || page >= p.pg.n_pages) {
      record(p.status, VARK_E_SHAPE);
      continue;
    }
    const int64_t in_page = row & ((1 << p.pg.log2_page) - 1);
    const int64_t hp = p.pg.page_heads > 1 ? h : 0;
    const int64_t at = (((page * p.pg.page_heads + hp) << p.pg.log2_page) + in_page) * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __stcs(reinterpret_cast<uint4*>(p.k_pages + at + ln.v[i] * 8), kw[r][i]);
      __stcs(reinterpret_cast<uint4*>(p.v_pages + at + ln.v[i] * 8), vw[r][i]);
    }
  }
}

// ------------------------------------------------------------------ host side
static int check_common(int dtype, int D, int norm, float eps) {
  if (dtype != VARK_BF16 && dtype != VARK_FP16) return VARK_E_ARG;
  if (norm < VARK_NORM_NONE || norm > VARK_NORM_L2 || !(eps >= 0.f)) return VARK_E_ARG;
  if (norm == VARK_NORM_L2 && eps > 0.f && eps < FLT_MIN) return VARK_E_ARG;      // 1 / eps would overflow
  if (D != 64 && D != 128) return VARK_E_SHAPE;
  return VARK_OK;
}

static int make_rotation(Rotation* r, const float* rope, int rope_len, int rope_dim, int pairs,
                         const int32_t* positions, int D) {
  *r = Rotation{nullptr, nullptr, 0, 0, 0};
  if (rope == nullptr && positions == nullptr) return VARK_OK;
  if (rope == nullptr || positions == nullptr) return VARK_E_ARG;
  if (rope_len < 1 || rope_dim < 16 || rope_dim > D || rope_dim % 16 != 0) return VARK_E_SHAPE;
  *r = Rotation{rope, positions, rope_len, rope_dim, pairs != 0};
  return VARK_OK;
}

// A tensor that is written over itself keeps its strides.
static bool in_place_alike(const RowTensor& t) {
  return t.src != t.dst || (t.ss[0] == t.ds[0] && t.ss[1] == t.ds[1] && t.ss[2] == t.ds[2]);
}

// Grid of warps over (token, block of heads).
static dim3 token_grid(int64_t tokens, int head_blocks) {
  const int warps = kRowThreads / 32;
  return dim3(unsigned((tokens + warps - 1) / warps), unsigned(head_blocks));
}
static int blocks_of(int heads, int per_block) { return (heads + per_block - 1) / per_block; }

}  // namespace paged
}  // namespace vark

using namespace vark;
using namespace vark::paged;

extern "C" int vark_qk_norm_rope(int dtype, const uint16_t* q, const int64_t* q_strides, uint16_t* q_out,
                                 const int64_t* q_out_strides, int Hq, const uint16_t* k, const int64_t* k_strides,
                                 uint16_t* k_out, const int64_t* k_out_strides, int Hk, int B, int T, int D, int norm,
                                 const float* q_weight, const float* k_weight, float eps, const float* rope,
                                 int rope_len, int rope_dim, int pairs, const int32_t* positions,
                                 int32_t* dev_status, void* stream) {
  if (!dev_status) return VARK_E_ARG;
  int rc = check_common(dtype, D, norm, eps);
  if (rc) return rc;
  if (B < 0 || T < 0) return VARK_E_SHAPE;
  if (B == 0 || T == 0) return check_device_sm100();       // empty tensors have no addresses to look at
  if ((!q && !k) || (q && (!q_strides || !q_out || !q_out_strides)) || (k && (!k_strides || !k_out || !k_out_strides)))
    return VARK_E_ARG;
  if ((q && Hq < 1) || (k && Hk < 1)) return VARK_E_SHAPE;
  if (Hq > 65536 || Hk > 65536 || int64_t(B) * T > INT32_MAX - kRowThreads) return VARK_E_SHAPE;
  NormRopeParams p;
  if ((rc = make_rotation(&p.rot, rope, rope_len, rope_dim, pairs, positions, D))) return rc;
  p.T = T;
  p.tokens = B * T;
  p.norm = norm;
  p.eps = eps;
  p.status = dev_status;
  const RowTensor none = {nullptr, nullptr, nullptr, {0, 0, 0}, {0, 0, 0}, 0};
  p.t[0] = p.t[1] = none;
  if (q) {
    const int64_t n[3] = {B, T, Hq};
    p.t[0] = RowTensor{q, q_out, q_weight, {0, 0, 0}, {0, 0, 0}, Hq};
    if (!take_strides(p.t[0].ss, q_strides, n, 3, 0) || !take_strides(p.t[0].ds, q_out_strides, n, 3, D) ||
        !rows_apart(p.t[0].ds, n, 3, D) || !aligned16(q) || !aligned16(q_out))
      return VARK_E_ALIGN;
    if (!in_place_alike(p.t[0])) return VARK_E_ARG;
  }
  if (k) {
    const int64_t n[3] = {B, T, Hk};
    p.t[1] = RowTensor{k, k_out, k_weight, {0, 0, 0}, {0, 0, 0}, Hk};
    if (!take_strides(p.t[1].ss, k_strides, n, 3, 0) || !take_strides(p.t[1].ds, k_out_strides, n, 3, D) ||
        !rows_apart(p.t[1].ds, n, 3, D) || !aligned16(k) || !aligned16(k_out))
      return VARK_E_ALIGN;
    if (!in_place_alike(p.t[1])) return VARK_E_ARG;
  }
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(rope)) return VARK_E_ALIGN;
  if ((rc = check_device_sm100())) return rc;
  p.q_blocks = blocks_of(p.t[0].heads, kQkHeads);
  const dim3 grid = token_grid(p.tokens, p.q_blocks + blocks_of(p.t[1].heads, kQkHeads));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == VARK_BF16)
    return D == 128 ? launch_early(norm_rope_kernel<VARK_BF16, 128>, grid, kRowThreads, 0, st, p)
                    : launch_early(norm_rope_kernel<VARK_BF16, 64>, grid, kRowThreads, 0, st, p);
  return D == 128 ? launch_early(norm_rope_kernel<VARK_FP16, 128>, grid, kRowThreads, 0, st, p)
                  : launch_early(norm_rope_kernel<VARK_FP16, 64>, grid, kRowThreads, 0, st, p);
}

extern "C" int vark_paged_append(int dtype, const uint16_t* k, const int64_t* k_strides, const uint16_t* v,
                                 const int64_t* v_strides, int64_t n_tokens, int B, int H, int D,
                                 const int32_t* cu_tokens, uint16_t* k_pages, uint16_t* v_pages, int64_t n_pages,
                                 int page_size, const int32_t* page_table, int max_pages, const int32_t* cache_len,
                                 int head_pages, int norm, const float* k_weight, float eps, const float* rope,
                                 int rope_len, int rope_dim, int pairs, const int32_t* positions,
                                 int32_t* dev_status, void* stream) {
  if (!dev_status) return VARK_E_ARG;
  int rc = check_common(dtype, D, norm, eps);
  if (rc) return rc;
  if (n_tokens < 0 || n_tokens > INT32_MAX - kRowThreads || B < 0 || B > (1 << 24) || H < 1 || H > 65536)
    return VARK_E_SHAPE;
  AppendParams p;
  if ((rc = make_pages(&p.pg, page_table, cache_len, n_pages, page_size, max_pages, H, head_pages))) return rc;
  if (n_tokens == 0 || B == 0) return check_device_sm100();       // empty tensors have no addresses to look at
  if (!k || !k_strides || !v || !v_strides || !cu_tokens || !k_pages || !v_pages || !page_table || !cache_len)
    return VARK_E_ARG;
  if ((rc = make_rotation(&p.rot, rope, rope_len, rope_dim, pairs, positions, D))) return rc;
  const int64_t extent[2] = {n_tokens, H};
  if (!take_strides(p.ks, k_strides, extent, 2, 0) || !take_strides(p.vs, v_strides, extent, 2, 0) || !aligned16(k) ||
      !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_weight) || !aligned16(rope))
    return VARK_E_ALIGN;
  if ((rc = check_device_sm100())) return rc;
  p.k = k; p.v = v;
  p.k_pages = k_pages; p.v_pages = v_pages;
  p.cu = cu_tokens;
  p.B = B;
  p.tokens = int(n_tokens);
  p.weight = k_weight;
  p.norm = norm;
  p.eps = eps;
  p.status = dev_status;
  const dim3 grid = token_grid(n_tokens, blocks_of(H, kKvHeads));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == VARK_BF16)
    return D == 128 ? launch_early(append_kernel<VARK_BF16, 128>, grid, kRowThreads, 0, st, p)
                    : launch_early(append_kernel<VARK_BF16, 64>, grid, kRowThreads, 0, st, p);
  return D == 128 ? launch_early(append_kernel<VARK_FP16, 128>, grid, kRowThreads, 0, st, p)
                  : launch_early(append_kernel<VARK_FP16, 64>, grid, kRowThreads, 0, st, p);
}
