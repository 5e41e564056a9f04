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
// Layout: D / 8 lanes hold a row, 8 channels (one 16-byte vector) each, so the
// sum of squares takes log2(D / 8) shuffles and the other half of a
// half-split pair is one lane's vector away.  A warp takes one token and up to
// 8 heads of it: all rows are loaded first, and the token's cosines and sines
// are read once for all of them.
#include "vark_paged.cuh"

namespace vark {
namespace paged {

constexpr int kRowThreads = 128;
constexpr int kHeadsPerWarp = 8;

struct Rotation {
  const float* table;       // [rope_len][2][dim / 2], or null
  const int32_t* positions; // [tokens]
  int len, dim, pairs;
};

// One lane's share of a token's rotation: which of its 8 channels turn, and
// the cosines and sines they need.
template <int LANES>
struct LaneRotation {
  float c[8], s[8];      // halves: 8 pairs; pairs: the first 4
  int partner;           // halves: lane (within the row) that holds the other half
  bool turns, first;     // first: this lane holds the a-half

  VARK_DEV void load(const Rotation& r, int pos, int li) {
    turns = r.table != nullptr && li * 8 < r.dim;
    first = true;
    partner = li;
    if (!turns) return;
    const int half = r.dim >> 1;
    const float* row = r.table + int64_t(pos) * r.dim;
    if (r.pairs) {
      const float4 cc = *reinterpret_cast<const float4*>(row + li * 4);
      const float4 ss = *reinterpret_cast<const float4*>(row + half + li * 4);
      c[0] = cc.x; c[1] = cc.y; c[2] = cc.z; c[3] = cc.w;
      s[0] = ss.x; s[1] = ss.y; s[2] = ss.z; s[3] = ss.w;
    } else {
      first = li * 8 < half;
      partner = first ? li + (half >> 3) : li - (half >> 3);
      const int j = first ? li * 8 : li * 8 - half;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 cc = *reinterpret_cast<const float4*>(row + j + e);
        const float4 ss = *reinterpret_cast<const float4*>(row + half + j + e);
        c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
        s[e] = ss.x; s[e + 1] = ss.y; s[e + 2] = ss.z; s[e + 3] = ss.w;
      }
    }
  }
};

// Norm and rotation of one row held by LANES lanes (every lane of the warp
// calls it; lanes without a row pass zeros).
template <int DT, int LANES>
VARK_DEV uint4 norm_rotate(uint4 w, int norm, float eps, bool weighted, const float (&wt)[8], const Rotation& rot,
                           const LaneRotation<LANES>& lr) {
  float x[8];
  unpack2<DT>(w.x, x[0], x[1]);
  unpack2<DT>(w.y, x[2], x[3]);
  unpack2<DT>(w.z, x[4], x[5]);
  unpack2<DT>(w.w, x[6], x[7]);
  if (norm != VARK_NORM_NONE) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = norm == VARK_NORM_RMS ? 1.f / sqrtf(ss * (1.f / (8 * LANES)) + eps) : 1.f / fmaxf(sqrtf(ss), eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= inv;
  }
  if (weighted) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= wt[e];
  }
  if (rot.table != nullptr) {
    if (rot.pairs) {
      if (lr.turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[2 * e], b = x[2 * e + 1];
          x[2 * e] = a * lr.c[e] - b * lr.s[e];
          x[2 * e + 1] = a * lr.s[e] + b * lr.c[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, x[e], lr.partner, LANES);
        if (lr.turns) x[e] = lr.first ? x[e] * lr.c[e] - o * lr.s[e] : o * lr.s[e] + x[e] * lr.c[e];
      }
    }
  }
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
}

// -1: the token is padding (not written); -2: position outside the table.
VARK_DEV int token_position(const Rotation& r, int64_t token) {
  if (r.table == nullptr) return 0;
  const int p = r.positions[token];
  return p < 0 ? -1 : (p >= r.len ? -2 : p);
}

VARK_DEV void load_weight(const float* w, int li, float (&wt)[8]) {
  if (w == nullptr) return;
  const float4 a = *reinterpret_cast<const float4*>(w + li * 8);
  const float4 b = *reinterpret_cast<const float4*>(w + li * 8 + 4);
  wt[0] = a.x; wt[1] = a.y; wt[2] = a.z; wt[3] = a.w;
  wt[4] = b.x; wt[5] = b.y; wt[6] = b.z; wt[7] = b.w;
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
  int T;
  int64_t tokens;          // B * T
  int blocks[2];           // warps a token takes for the queries' heads, the keys'
  int norm;
  float eps;
  Rotation rot;
  int32_t* status;
};

template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kHeadsPerWarp / kRows;
  const int lane = threadIdx.x & 31, li = lane % kLanes, sub = lane / kLanes;
  const int per_token = p.blocks[0] + p.blocks[1];
  const int64_t unit = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = unit / per_token;
  if (token >= p.tokens) return;
  int blk = int(unit - token * per_token);
  const int which = blk >= p.blocks[0];
  if (which) blk -= p.blocks[0];
  const RowTensor& t = p.t[which];
  const int pos = token_position(p.rot, token);
  if (pos < 0) {
    if (pos == -2 && lane == 0) record(p.status, VARK_E_SHAPE);
    return;
  }
  const int64_t b = token / p.T, i = token - b * p.T;
  const uint16_t* src = t.src + b * t.ss[0] + i * t.ss[1] + li * 8;
  uint16_t* dst = t.dst + b * t.ds[0] + i * t.ds[1] + li * 8;
  const int h0 = blk * kHeadsPerWarp + sub;
  uint4 v[kIters];
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    v[r] = h < t.heads ? ld_stream(src + h * t.ss[2]) : make_uint4(0u, 0u, 0u, 0u);
  }
  LaneRotation<kLanes> lr;
  lr.load(p.rot, pos, li);
  float wt[8];
  load_weight(t.weight, li, wt);
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    const uint4 o = norm_rotate<DT, kLanes>(v[r], p.norm, p.eps, t.weight != nullptr, wt, p.rot, lr);
    if (h < t.heads) *reinterpret_cast<uint4*>(dst + h * t.ds[2]) = o;
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
  int B;
  int64_t tokens;
  int blocks;              // warps a token takes
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

template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kHeadsPerWarp / kRows;
  const int lane = threadIdx.x & 31, li = lane % kLanes, sub = lane / kLanes;
  const int64_t unit = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = unit / p.blocks;
  if (token >= p.tokens) return;
  const int h0 = int(unit - token * p.blocks) * kHeadsPerWarp + sub;
  const int pos = token_position(p.rot, token);
  const int b = find_sequence(p.cu, p.B, token, lane);
  if (b < 0 || b >= p.B || pos == -1) return;   // outside every sequence, or padding
  if (pos == -2) {
    if (lane == 0) record(p.status, VARK_E_SHAPE);
    return;
  }
  const int first = p.cu[b], n = p.cu[b + 1] - first;
  if (token - first >= n) return;               // tables that do not ascend
  const uint16_t* ks = p.k + token * p.ks[0] + li * 8;
  const uint16_t* vs = p.v + token * p.vs[0] + li * 8;
  uint4 kv[kIters], vv[kIters];
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    kv[r] = vv[r] = make_uint4(0u, 0u, 0u, 0u);
    if (h < p.pg.heads) {
      kv[r] = ld_stream(ks + h * p.ks[1]);
      vv[r] = ld_stream(vs + h * p.vs[1]);
    }
  }
  LaneRotation<kLanes> lr;
  lr.load(p.rot, pos, li);
  float wt[8];
  load_weight(p.weight, li, wt);
#pragma unroll
  for (int r = 0; r < kIters; ++r) {
    const int h = h0 + r * kRows;
    const uint4 o = norm_rotate<DT, kLanes>(kv[r], p.norm, p.eps, p.weight != nullptr, wt, p.rot, lr);
    if (h >= p.pg.heads) continue;
    const int64_t e = int64_t(b) * p.pg.table_heads + (p.pg.table_heads > 1 ? h : 0);
    const int64_t row = int64_t(p.pg.len[e]) - n + (token - first);
    if (row < 0) continue;                      // the cache holds only the chunk's last len rows
    const int64_t pi = row >> p.pg.log2_page;
    const int64_t page = pi < p.pg.max_pages ? p.pg.table[e * p.pg.max_pages + pi] : -1;
    if (page < 0 || page >= p.pg.n_pages) {
      record(p.status, VARK_E_SHAPE);
      continue;
    }
    const int64_t in_page = row & ((1 << p.pg.log2_page) - 1);
    const int64_t hp = p.pg.page_heads > 1 ? h : 0;
    const int64_t at = ((((page * p.pg.page_heads + hp) << p.pg.log2_page) + in_page) * D) + li * 8;
    *reinterpret_cast<uint4*>(p.k_pages + at) = o;
    *reinterpret_cast<uint4*>(p.v_pages + at) = vv[r];
  }
}

// ------------------------------------------------------------------ host side
static int check_common(int dtype, int D, int norm, float eps) {
  if (dtype != VARK_BF16 && dtype != VARK_FP16) return VARK_E_ARG;
  if (norm < VARK_NORM_NONE || norm > VARK_NORM_L2 || !(eps >= 0.f)) return VARK_E_ARG;
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


static int launch_units(int64_t units, unsigned* grid) {
  const int64_t g = (units + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (g > INT32_MAX) return VARK_E_SHAPE;
  *grid = unsigned(g);
  return VARK_OK;
}

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
  if (!dev_status || (!q && !k)) return VARK_E_ARG;
  if (q && (!q_strides || !q_out || !q_out_strides)) return VARK_E_ARG;
  if (k && (!k_strides || !k_out || !k_out_strides)) return VARK_E_ARG;
  int rc = check_common(dtype, D, norm, eps);
  if (rc) return rc;
  if (B < 0 || T < 0 || (q && Hq < 1) || (k && Hk < 1)) return VARK_E_SHAPE;
  if (Hq > 65536 || Hk > 65536 || int64_t(B) * T > (int64_t(1) << 40)) return VARK_E_SHAPE;
  NormRopeParams p;
  if ((rc = make_rotation(&p.rot, rope, rope_len, rope_dim, pairs, positions, D))) return rc;
  p.T = T > 0 ? T : 1;
  p.tokens = int64_t(B) * T;
  p.norm = norm;
  p.eps = eps;
  p.status = dev_status;
  const RowTensor none = {nullptr, nullptr, nullptr, {0, 0, 0}, {0, 0, 0}, 0};
  p.t[0] = p.t[1] = none;
  if (q) {
    const int64_t n[3] = {B, T, Hq};
    p.t[0] = RowTensor{q, q_out, q_weight, {0, 0, 0}, {0, 0, 0}, Hq};
    if (!take_strides(p.t[0].ss, q_strides, n, 3) || !take_strides(p.t[0].ds, q_out_strides, n, 3) ||
        !aligned16(q) || !aligned16(q_out))
      return VARK_E_ALIGN;
  }
  if (k) {
    const int64_t n[3] = {B, T, Hk};
    p.t[1] = RowTensor{k, k_out, k_weight, {0, 0, 0}, {0, 0, 0}, Hk};
    if (!take_strides(p.t[1].ss, k_strides, n, 3) || !take_strides(p.t[1].ds, k_out_strides, n, 3) ||
        !aligned16(k) || !aligned16(k_out))
      return VARK_E_ALIGN;
  }
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(rope)) return VARK_E_ALIGN;
  if ((rc = check_device_sm100())) return rc;
  if (p.tokens == 0) return VARK_OK;
  for (int i = 0; i < 2; ++i) p.blocks[i] = (p.t[i].heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  unsigned grid;
  if ((rc = launch_units(p.tokens * (p.blocks[0] + p.blocks[1]), &grid))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == VARK_BF16) {
    if (D == 128) norm_rope_kernel<VARK_BF16, 128><<<grid, kRowThreads, 0, st>>>(p);
    else norm_rope_kernel<VARK_BF16, 64><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    if (D == 128) norm_rope_kernel<VARK_FP16, 128><<<grid, kRowThreads, 0, st>>>(p);
    else norm_rope_kernel<VARK_FP16, 64><<<grid, kRowThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? VARK_OK : VARK_E_CUDA;
}

extern "C" int vark_paged_append(int dtype, const uint16_t* k, const int64_t* k_strides, const uint16_t* v,
                                 const int64_t* v_strides, int64_t n_tokens, int B, int H, int D,
                                 const int32_t* cu_tokens, uint16_t* k_pages, uint16_t* v_pages, int64_t n_pages,
                                 int page_size, const int32_t* page_table, int max_pages, const int32_t* cache_len,
                                 int head_pages, int norm, const float* k_weight, float eps, const float* rope,
                                 int rope_len, int rope_dim, int pairs, const int32_t* positions,
                                 int32_t* dev_status, void* stream) {
  if (!k || !k_strides || !v || !v_strides || !cu_tokens || !k_pages || !v_pages || !page_table || !cache_len ||
      !dev_status)
    return VARK_E_ARG;
  int rc = check_common(dtype, D, norm, eps);
  if (rc) return rc;
  if (n_tokens < 0 || n_tokens > INT32_MAX || B < 0 || B > (1 << 24) || H < 1 || H > 65536) return VARK_E_SHAPE;
  AppendParams p;
  if ((rc = make_rotation(&p.rot, rope, rope_len, rope_dim, pairs, positions, D))) return rc;
  if ((rc = make_pages(&p.pg, page_table, cache_len, n_pages, page_size, max_pages, H, head_pages))) return rc;
  const int64_t extent[2] = {n_tokens, H};
  if (!take_strides(p.ks, k_strides, extent, 2) || !take_strides(p.vs, v_strides, extent, 2) || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_weight) || !aligned16(rope))
    return VARK_E_ALIGN;
  if ((rc = check_device_sm100())) return rc;
  if (n_tokens == 0 || B == 0) return VARK_OK;
  p.k = k; p.v = v;
  p.k_pages = k_pages; p.v_pages = v_pages;
  p.cu = cu_tokens;
  p.B = B;
  p.tokens = n_tokens;
  p.weight = k_weight;
  p.norm = norm;
  p.eps = eps;
  p.status = dev_status;
  p.blocks = (H + kHeadsPerWarp - 1) / kHeadsPerWarp;
  unsigned grid;
  if ((rc = launch_units(n_tokens * p.blocks, &grid))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == VARK_BF16) {
    if (D == 128) append_kernel<VARK_BF16, 128><<<grid, kRowThreads, 0, st>>>(p);
    else append_kernel<VARK_BF16, 64><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    if (D == 128) append_kernel<VARK_FP16, 128><<<grid, kRowThreads, 0, st>>>(p);
    else append_kernel<VARK_FP16, 64><<<grid, kRowThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? VARK_OK : VARK_E_CUDA;
}
