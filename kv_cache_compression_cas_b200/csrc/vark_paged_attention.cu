// Attention of a chunk of new tokens over a paged cache (vark_paged_attention).
//
// Mathematics: query row i of head h sees keys j < lim_i; with x_j = tau[h]
// (q_i . k_j) / sqrt(D) the output is sum_j 2^(x'_j - m) v_j / l, x' = x log2 e,
// m the running maximum and l = sum_j 2^(x'_j - m): one pass over the keys.
//
// The G query heads of a kv head share its keys, so the G * n rows of a
// sequence's n tokens (token-major: row = token * G + head) are cut into tiles
// of R rows: an item is (sequence, kv head, row tile).  Work is split along the
// keys as well: all items are laid end to end, each as long as it costs, and
// every CTA takes an equal share of the whole, so one long cache spreads over
// the device and a ragged batch leaves no CTA with the longest sequence (a few
// short items of many rows stay whole: kCutTiles).  An item that falls
// into several shares leaves one partial (o, m, l) per CTA in the workspace; a
// second, small kernel joins them.  Lengths live on the device: every CTA
// finds its share with one scan over the sequence table.
#include <atomic>
#include <cstdlib>

#include "vark_paged.cuh"
#include "vark_paged_plan.cuh"

namespace vark {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;       // log2: a running maximum may lag by this much
// log2: how far below a row's maximum its probabilities' reference lies.  They
// are summed in fp32 and rounded to the cache's type for P V, whose MMAs take 16
// bits.  bf16 has fp32's range; of fp16, below 2^-14 a step is 2^-24 and below
// 2^-25 nothing is left, so the reference lies where the largest come to 2^15
// (with the lag): a probability is then off by 2^-32 of the largest at most,
// where it was 2^-25, at which 65536 keys 17 below one in the logits came out
// 44% too heavy and 18 below were lost.
template <int DT>
constexpr float kLift = DT == VARK_FP16 ? 7.0f : 0.0f;

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;              // [N][Hq] or null
  int64_t qs[2], os[2];    // token, head strides (elements)
  Pages pg;
  const int32_t* cu;       // [B + 1]
  const float* tau;        // [Hq] or null
  int64_t N;
  int B, G, Hq, causal;
  FastDiv by_group, by_heads;   // / G, / kv heads
  int tokens_per_tile;     // R / G
  int tile_step;           // kUnit R / G: weight from a row tile to the next under a causal mask
  float scale_log2;        // log2(e) / sqrt(D)
  float* part_o;           // [kCtas][2][R][D]
  float* part_ml;          // [kCtas][2][R][2]
  int32_t* status;
  uint64_t wait_limit_ns;
  int withhold;            // test hook: key tiles a CTA loads before it stops (-1: all)

  // Row e of the length table.  Lengths and token offsets that do not fit the
  // arguments leave it without work and are recorded.
  template <int R, int KT>
  VARK_DEV Entry entry(int e) const {
    Entry x;
    const int b = pg.table_heads > 1 ? by_heads(e) : e;
    x.first = __ldcg(cu + b);     // (past L1: the join plans before it waits for the kernels ahead of it)
    const int end = __ldcg(cu + b + 1);
    x.len = __ldcg(pg.len + e);
    if (x.first < 0 || end < x.first || end > N || x.len < 0 || (x.len - 1) >> pg.log2_page >= pg.max_pages) {
      record(status, VARK_E_SHAPE);
      x.first = x.n = x.len = 0;
    } else {
      x.n = end - x.first;
    }
    x.weigh<R, KT>(*this);
    return x;
  }
};

// ------------------------------------------------------------------ the plan
// The arithmetic is in vark_paged_plan.cuh; here the scan over the tables.


// Running sum over the lanes of a warp.
template <typename T>
VARK_DEV T lane_sums(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// From the warps' sums: what lies before this warp, and all of it.  (By lanes:
// a loop over the warps, unrolled, is 100 instructions that run once, and those
// cost most by being fetched.)
template <int WARPS, typename T>
VARK_DEV void warp_sums(const T* of, int warp, int lane, T& before, T& total) {
  const T own = lane < WARPS ? of[lane] : T(0);
  const T incl = lane_sums(own, lane);
  total = __shfl_sync(0xffffffffu, incl, WARPS - 1);
  before = __shfl_sync(0xffffffffu, incl - own, warp);
}

// Scan over the entries by the whole block: the share of CTA `cta`, and where
// its first unit (and with LAST its last one) lies.
template <int R, int KT, int THREADS, bool LAST>
VARK_DEV Share find_share(const AttnParams& p, int cta) {
  constexpr int kWarps = THREADS / 32;
  constexpr int64_t kTile = int64_t(kUnit) * KT;
  constexpr bool kMayCount = R == kTileR;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int warp_longest[kWarps], warp_items[kWarps];
  __shared__ Share::Place found[2];
  const int E = p.B * p.pg.table_heads;
  const int chunk = (E + THREADS - 1) / THREADS;
  const int e0 = min(E, int(threadIdx.x) * chunk), e1 = min(E, e0 + chunk);
  int64_t sum = 0, items = 0, longest = 0;
  Entry x = {};
  for (int e = e0; e < e1; ++e) {
    x = p.entry<R, KT>(e);
    sum += x.units();
    if (kMayCount) {
      items += int64_t(x.heads) * x.row_tiles;
      longest = max(longest, x.longest());
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = lane_sums(sum, lane);
  if (kMayCount) {
    const int tiles = __reduce_max_sync(0xffffffffu, int((longest + kTile - 1) / kTile));
    if (lane == 0) warp_longest[warp] = tiles;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  Share s;
  int64_t before, total;
  warp_sums<kWarps>(warp_sum, warp, lane, before, total);
  bool one_each = false;             // every item weighs one unit: none is cut
  if (kMayCount) {
    const int tiles = __reduce_max_sync(0xffffffffu, lane < kWarps ? warp_longest[lane] : 0);
    if (worth_whole<KT>(tiles, total)) {        // (the same for every thread)
      const int own = int(min(items, int64_t(kCtas + 1)));
      const int incl_items = lane_sums(own, lane);
      if (lane == 31) warp_items[warp] = incl_items;
      __syncthreads();
      int before_items, all_items;
      warp_sums<kWarps>(warp_items, warp, lane, before_items, all_items);
      if (all_items <= kCtas) {
        one_each = true;
        total = all_items;
        before = before_items;
        sum = own;
        incl = incl_items;
        x.count_items();
      }
    }
  }
  s.split(total);
  s.u0 = s.u1 = 0;
  if (cta >= s.ctas) return s;   // the same for every thread
  s.u0 = s.begin(cta);
  s.u1 = s.begin(cta + 1);
  const int64_t from = before + incl - sum;
#pragma unroll
  for (int k = 0; k < (LAST ? 2 : 1); ++k) {
    const int64_t want = k ? s.u1 - 1 : s.u0;
    if (want < from || want >= from + sum) continue;
    int64_t base = from;
    for (int e = e0; e < e1; ++e) {
      if (chunk > 1) {                                // (else it is the one just read)
        x = p.entry<R, KT>(e);
        if (one_each) x.count_items();
      }
      const int64_t w = x.units();
      if (want < base + w) {
        found[k] = Share::Place{e, base, x};
        break;
      }
      base += w;
    }
  }
  __syncthreads();
  s.first = found[0];
  if (LAST) s.last = found[1];
  return s;
}

struct RowAt {
  int token, head;         // token of the batch, query head; token < 0: no such row
  int limit;               // keys it sees
};
template <int R, int KT>
VARK_DEV RowAt row_at(const AttnParams& p, const Segments<R, KT>& s, int r) {
  RowAt a;
  const int row = s.tile * R + r;
  const int t = p.by_group(row);
  a.head = s.h * p.G + (row - t * p.G);
  a.token = t < s.x.n ? s.x.first + t : -1;
  a.limit = t >= s.x.n ? 0 : p.causal ? s.x.len - s.x.n + t + 1 : s.x.len;
  return a;
}

// Writes 8 channels of a finished row (o not yet divided by l).
template <int DT>
VARK_DEV void store_row8(const AttnParams& p, const RowAt& a, int d0, const float (&o)[8], float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;    // no key: zeros
  uint4 w;
  w.x = pack2<DT>(o[0] * inv, o[1] * inv);
  w.y = pack2<DT>(o[2] * inv, o[3] * inv);
  w.z = pack2<DT>(o[4] * inv, o[5] * inv);
  w.w = pack2<DT>(o[6] * inv, o[7] * inv);
  *reinterpret_cast<uint4*>(p.out + a.token * p.os[0] + a.head * p.os[1] + d0) = w;
  if (d0 == 0 && p.lse != nullptr)
    p.lse[int64_t(a.token) * p.Hq + a.head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ tiles kernel
// Many rows a kv head (prompt chunks, scales): bound by the tensor cores.  A
// CTA works on 256 rows as two tiles of 128 (A, B) that see the same key tiles,
// so every key tile is loaded once for both.  Warp 0 loads key and value
// tiles of 128 rows by TMA, one box per page, into one ring of slots (K_0, V_0,
// K_1, V_1, ...); warps 2 and 3 bring the queries of A and B, a segment ahead of
// their use; warp 1 issues the MMAs PV_A(j-1), S_A(j), PV_B(j-1), S_B(j),
// so the softmax of one tile overlaps the products of the other; warps 4-7 and
// 8-11 are the softmax of A and B, one thread per row (TMEM lane).  S is read
// from tensor memory, and P written back over its first 64 columns in the type
// of the values, where the PV MMA takes it as its A operand.  O stays in tensor
// memory and is rescaled only when a row's maximum grows by more than 2^8.
// The MMA warp runs its loop with all lanes and only predicates the MMAs:
// descriptors and addresses then stay warp-uniform.
//
// Measured (32 heads of 128 over 8 kv heads, bf16), call after call, at the power
// limit: a chunk of 2048 tokens over 16384 cached rows 566 to 585 us, 1.0
// PFLOP/s; 8 prompts of 333 to 4099 tokens 501 to 512 us (one call after a rest,
// while the clock holds: 503 and 478).  A pair of tiles takes 3500 cycles for 128 keys: 2050 of MMAs, whose
// S products read 128 B/clk of shared memory, and as much of exp2 on the two
// softmax warps of an SM quarter.  What ties them is S -> softmax -> PV -> S.
// Keys in halves with S a half ahead cut that chain and cost 535 and 495 us:
// N = 64 products read 192 B/clk, and barriers come twice as often.  P in two
// chunks 556 for 521, a share of the exponentials as polynomials 4 to 10% more.
// An item costs 10000 cycles besides its key tiles: prompts feel it.
// TMEM: S_A [0,128) S_B [128,256) O_A [256,256+D) O_B [256+D,256+2D).
//
// An MMA cuts its products off 2^-25 below the sum that it adds them to
// (measured: a key of 2^-25 of the sum counts in full, one of 2^-26 not at all),
// so n keys can lose 1.25 n 2^-25 of an output while l keeps them: of 2^20 keys
// of equal weight 0.6% of it, always towards zero.  Every kSumTiles key tiles
// the softmax threads therefore add O to an fp32 row in the workspace (the slot
// of the segment's partial result, which nothing else uses meanwhile) and begin
// it anew: 0.12% at most, 0.02% at equal weights.  That takes as long as 4 key
// tiles; every 128 tiles 2.5% of the chunk above.
constexpr int kSumTiles = 256;
constexpr int kTileThreads = 384;
constexpr int kMaxSmem = 232448;

VARK_DEV uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// The MMAs and commits of the thread whose `lead` is 1 (all lanes pass by).
VARK_DEV void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
VARK_DEV void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
VARK_DEV void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Instruction descriptor, kind::f16: A and B of type DT, fp32 accumulator.
template <int DT>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool b_mn_major) {
  return (1u << 4) | (DT == VARK_BF16 ? (1u << 7) | (1u << 10) : 0u) | (uint32_t(b_mn_major) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

template <int D>
struct TileSmem {
  static constexpr int kPanel = 128 * 128;            // 128 rows x 64 channels
  static constexpr int kTile = (D / 64) * kPanel;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kQ = 0;                        // [2 tiles]
  static constexpr int kRing = kQ + 2 * kTile;        // [kSlots]
  static constexpr int kStage = kRing + kSlots * kTile;   // [8 softmax warps] 32 rows of 128 bytes on their way out
  static constexpr int kStageBytes = 32 * 128;
  static constexpr int kBar = kStage + 8 * kStageBytes;
  static constexpr int kFull = 0, kEmpty = kSlots;    // barrier indices
  static constexpr int kQFull = 2 * kSlots, kQFree = kQFull + 2, kS = kQFree + 2, kP = kS + 2, kO = kP + 2;
  static constexpr int kDrain = kO + 2, kNumBars = kDrain + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;   // tmem base, abort flag
  static constexpr int kSeg = kMisc + 16;             // [warps 1-3, 8 softmax warps] segment, out of their registers
  static constexpr int kSegBytes = 112;
  static constexpr int kAlloc = kSeg + 11 * kSegBytes;
  static_assert(kAlloc + 1024 <= kMaxSmem, "shared memory");
};

// A place in the ring: slot i % kSlots, with the parity of its round.
template <int SLOTS>
struct RingAt {
  int slot, phase;
  VARK_DEV void skip(int n) {
    slot += n;
    if (slot >= SLOTS) {
      slot -= SLOTS;
      phase ^= 1;
    }
  }
};

// Key tiles of a segment that some row of the item sees.
template <int R, int KT>
VARK_DEV int seen_tiles(const AttnParams& p, const Segments<R, KT>& s) {
  return max(0, min(s.k1, (s.limit(p) + KT - 1) / KT) - s.k0);
}

// The loading warp of both kernels: the key and value tiles of a share's
// segments, in order, into the ring of layout L (kRing, kTile, kPanel, kSlots,
// kBar, kFull, kEmpty).  Lane i loads the tile's i-th box: 128 rows, or a page
// where pages are smaller, whose number it asked for one tile ahead.
template <int D, int R, typename L>
VARK_DEV void load_tiles(const AttnParams& p, const Share& share, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                         uint32_t sbase, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + L::kBar + 8u * uint32_t(i); };
  const int box_log2 = min(p.pg.log2_page, 7);
  const int boxes = kTileKT >> box_log2;
  const int page_mask = (1 << p.pg.log2_page) - 1;
  Segments<R, kTileKT> sg;
  sg.start(p, share);
  RingAt<L::kSlots> at = {0, 0};
  int issued = 0;
  bool ok = true;
  while (ok && sg.next(p)) {
    const int nt = seen_tiles(p, sg);
    const int32_t* table = p.pg.table + int64_t(sg.e) * p.pg.max_pages;
    const int head_row = (p.pg.page_heads > 1 ? sg.h : 0) << p.pg.log2_page;
    int key = sg.k0 * kTileKT + (lane << box_log2);      // first key of this lane's box
    auto page_of = [&](int k) { return lane < boxes && k < sg.x.len ? table[k >> p.pg.log2_page] : 0; };
    int page = nt > 0 ? page_of(key) : 0;
    for (int j = 0; ok && j < nt; ++j) {
      const int next_page = j + 1 < nt ? page_of(key + kTileKT) : 0;
      if (page < 0 || page >= p.pg.n_pages) {
        record(p.status, VARK_E_SHAPE);
        page = 0;           // in bounds; the call's outputs are void
      }
      const bool mine = lane < boxes && key < sg.x.len;
      const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, mine))) << (box_log2 + (D == 128 ? 8 : 7));
      const int row = head_row + (key & page_mask);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (issued / 2 == p.withhold) ok = false;        // test hook: this tile never arrives
        ok = ok && (issued < L::kSlots || mbar_wait(bar(L::kEmpty + at.slot), uint32_t(at.phase ^ 1), abort_flag,
                                                    p.status, p.wait_limit_ns));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t full = bar(L::kFull + at.slot);
        const uint32_t dst = sbase + L::kRing + at.slot * L::kTile + (lane << (box_log2 + 7));
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (mine) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * L::kPanel, which ? &tm_v : &tm_k, full, c * 64, row, page);
        }
        ++issued;
        at.skip(1);
      }
      page = next_page;
      key += kTileKT;
    }
  }
  // Every load has landed before the CTA exits (at once unless a wait gave up).
  volatile int no_abort = 0;
  for (int i = max(0, issued - L::kSlots); i < issued; ++i)
    mbar_wait(bar(L::kFull + i % L::kSlots), (i / L::kSlots) & 1, &no_abort, nullptr);
}

VARK_DEV uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 16 bytes to shared memory without a register, zeros for `bytes` = 0.
VARK_DEV void copy_async16(uint32_t dst, const uint16_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
VARK_DEV void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Steps a warp's segment in shared memory.
template <int R, int KT>
VARK_DEV bool next_segment(const AttnParams& p, Segments<R, KT>& sg) {
  __syncwarp();
  Segments<R, KT> next = sg;          // every lane steps a copy in registers
  const bool more = next.next(p);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) sg = next;
  __syncwarp();
  return more;
}

template <int DT, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ AttnParams p) {
  using L = TileSmem<D>;
  using Seg = Segments<kTileR, kTileKT>;
  using Ring = RingAt<L::kSlots>;
  static_assert(sizeof(Seg) <= L::kSegBytes && sizeof(Seg) % 8 == 0 && L::kSeg % 8 == 0, "segment");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {      // (the swizzle counts on the alignment; there is no room to move the base)
    record(p.status, VARK_E_CUDA);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * uint32_t(i); };
  auto wait = [&](int i, int phase) {
    return mbar_wait(bar(i), uint32_t(phase), abort_flag, p.status, p.wait_limit_ns);
  };
  // One answer for a warp: a wait that one lane sees completed and another given
  // up must not part them.
  auto wait_all = [&](int i, int phase) { return __all_sync(0xffffffffu, wait(i, phase)) != 0; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bar(L::kFull + i), 1);
      mbar_init(bar(L::kEmpty + i), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(L::kQFull + x), 1);
      mbar_init(bar(L::kQFree + x), 1);
      mbar_init(bar(L::kS + x), 1);
      mbar_init(bar(L::kP + x), 4);
      mbar_init(bar(L::kO + x), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_wait();
  grid_release();           // only now: the join plans before it waits, so what wrote the tables has ended
  const Share share = find_share<kTileR, kTileKT, kTileThreads, false>(p, blockIdx.x);   // syncs the block
  if (share.u0 == share.u1) return;
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    setmaxnreg_dec56();
    if (warp == 0) {
      load_tiles<D, kTileR, L>(p, share, tm_k, tm_v, sbase, abort_flag);
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issue
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc_s = idesc_of<DT>(128, 128, false);
      constexpr uint32_t idesc_o = idesc_of<DT>(128, D, true);
      const uint64_t dq = smem_desc_sw128(sbase + L::kQ, 16, 1024);
      const uint64_t dk = smem_desc_sw128(sbase + L::kRing, 16, 1024);
      const uint64_t dv = smem_desc_sw128(sbase + L::kRing, L::kPanel, 1024);
      auto issue_s = [&](int x, int slot) {
        const uint64_t a = dq + uint32_t(x * (L::kTile >> 4)), b = dk + uint32_t(slot * (L::kTile >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * L::kPanel + (k & 3) * 32) >> 4;
          mma_ss(lead, tmem + x * 128, a + off, b + off, idesc_s, k > 0);
        }
      };
      auto issue_pv = [&](int x, int slot, uint32_t acc) {
        const uint64_t b = dv + uint32_t(slot * (L::kTile >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts(lead, tmem + 256 + x * D, tmem + x * 128 + k * 8, b + k * (2048 >> 4), idesc_o, k > 0 ? 1u : acc);
      };
      Seg& sg = *reinterpret_cast<Seg*>(smem + L::kSeg);
      if (lane == 0) sg.start(p, share);
      Ring kr = {0, 0}, vr = {1, 0};
      int q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      bool ok = true;
      while (ok && next_segment(p, sg)) {
        const int nt = seen_tiles(p, sg);
        const int n_act = sg.x.n * p.G - sg.tile * kTileR > 128 ? 2 : 1;
        for (int j = 0; ok && j <= nt && nt > 0; ++j) {
          if (j < nt) ok = wait(L::kFull + kr.slot, kr.phase);
          if (ok && j > 0) ok = wait(L::kFull + vr.slot, vr.phase);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x >= n_act || !ok) break;
            if (j > 0) {
              ok = wait(L::kP + x, p_phase[x]);
              if (!ok) break;
              p_phase[x] ^= 1;
              tc_fence_after();
              issue_pv(x, vr.slot, j > 1);
            } else {
              ok = wait(L::kQFull + x, q_phase[x]);
              if (!ok) break;
              q_phase[x] ^= 1;
              tc_fence_after();
            }
            if (j < nt) {
              issue_s(x, kr.slot);
              commit(lead, bar(L::kS + x));
              if (j == nt - 1) commit(lead, bar(L::kQFree + x));
            } else {
              commit(lead, bar(L::kO + x));
            }
          }
          // (asked once a key tile, behind the MMAs: a lane that gave up above
          // left nothing that the others wait for in lockstep)
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (j > 0) {
            commit(lead, bar(L::kEmpty + vr.slot));
            vr.skip(2);
          }
          if (j < nt) {
            commit(lead, bar(L::kEmpty + kr.slot));
            kr.skip(2);
          }
        }
      }
      // All MMAs are done before tensor memory is released.
      commit(lead, bar(L::kDrain));
      volatile int no_abort = 0;
      mbar_wait(bar(L::kDrain), 0, &no_abort, nullptr);
    } else {
      // -------------------------------------------------------- queries
      // Tile x's 128 rows, 128-byte swizzled, D / 8 lanes a row.  Under a
      // negative temperature the query's sign is turned instead, so the
      // largest score gives the largest logit; under 0, and where the factor of
      // the scores rounds to 0, the query is 0.
      constexpr int kRowLanes = D / 8, kRowsAt = 32 / kRowLanes;
      const int x = warp - 2;
      const uint32_t sq = sbase + L::kQ + x * L::kTile;
      auto chunk_at = [&](int w, int c) { return sq + (c >> 3) * L::kPanel + w * 128 + (((c & 7) ^ (w & 7)) << 4); };
      Seg& sg = *reinterpret_cast<Seg*>(smem + L::kSeg + (warp - 1) * L::kSegBytes);
      if (lane == 0) sg.start(p, share);
      int uses = 0;
      bool ok = true;
      while (ok && next_segment(p, sg)) {
        if (seen_tiles(p, sg) == 0 || (x == 1 && sg.x.n * p.G - sg.tile * kTileR <= 128)) continue;
        if (uses > 0) ok = wait_all(L::kQFree + x, (uses - 1) & 1);
        if (!ok) break;
        ++uses;
        bool turned = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const RowAt row = row_at(p, sg, x * 128 + q * 32 + lane);
          const float tau = p.tau != nullptr && row.token >= 0 ? p.tau[row.head] : 1.f;
          const bool none = row.token < 0 || p.scale_log2 * tau == 0.f;
          const int64_t off = none ? -1 : row.token * p.qs[0] + row.head * p.qs[1];
          turned |= tau < 0.f;
#pragma unroll 4
          for (int it = 0; it < 32 / kRowsAt; ++it) {
            const int w = it * kRowsAt + lane / kRowLanes, c = lane % kRowLanes;
            const int64_t from = __shfl_sync(0xffffffffu, off, w);
            copy_async16(chunk_at(q * 32 + w, c), p.q + (from < 0 ? 0 : from) + c * 8, from < 0 ? 0 : 16);
          }
        }
        copy_async_wait();
        __syncwarp();
        if (__any_sync(0xffffffffu, turned)) {
          for (int q = 0; q < 4; ++q) {
            const RowAt row = row_at(p, sg, x * 128 + q * 32 + lane);
            if (row.token < 0 || !(p.tau[row.head] < 0.f)) continue;
            for (int c = 0; c < kRowLanes; ++c) {
              uint4 v = ld_shared_v4(chunk_at(q * 32 + lane, c));
              v.x ^= 0x80008000u; v.y ^= 0x80008000u; v.z ^= 0x80008000u; v.w ^= 0x80008000u;
              st_shared_v4(chunk_at(q * 32 + lane, c), v);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kQFull + x));
      }
    }
  } else {
    setmaxnreg_inc224();
    // ---------------------------------------------------------- softmax
    const int x = (warp >> 2) - 1;
    const int r = threadIdx.x - 128 * (x + 1);          // row within the tile = TMEM lane
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_base;
    const uint32_t tO = tmem + 256 + x * D + lane_base;
    int s_phase = 0, o_phase = 0;
    Ring vr = {1, 0};
    bool ok = true;
    Seg& sg = *reinterpret_cast<Seg*>(smem + L::kSeg + (warp - 1) * L::kSegBytes);
    if (lane == 0) sg.start(p, share);
    // This row's part of a segment; the next one's is found while the last
    // products of the one before are still running.
    struct Work {
      RowAt row;
      int nt, seen, held;    // key tiles; keys from the first tile on that the row sees, that the cache holds
      int seen_min;          // over the warp's rows
      float qk2;             // (the temperature's sign is in the query, as is a zero)
      bool whole;
      int slot;
    } cur;
    auto take = [&](Work& w) {
      do {
        if (!next_segment(p, sg)) return false;
      } while (x == 1 && sg.x.n * p.G - sg.tile * kTileR <= 128);      // tile B may be empty
      w.row = row_at(p, sg, x * 128 + r);
      w.qk2 = p.scale_log2;
      if (p.tau != nullptr && w.row.token >= 0) {
        const float f = w.qk2 * fabsf(p.tau[w.row.head]);
        w.qk2 = f == 0.f ? 1.f : f;
      }
      w.nt = seen_tiles(p, sg);
      // (a row that does not exist needs no mask: nothing reads what it makes)
      w.seen = (w.row.token < 0 ? (1 << 30) : w.row.limit) - sg.k0 * kTileKT;
      w.held = sg.x.len - sg.k0 * kTileKT;
      w.seen_min = __reduce_min_sync(0xffffffffu, w.seen);
      w.whole = sg.whole();
      w.slot = part_slot(blockIdx.x, sg.k0) * kTileR + x * 128 + r;
      return true;
    };
    // O and the row in the workspace (see kSumTiles; its reference in part_ml): both
    // added up in the row (`save`; O is left at 0), or in O.
    auto move_sum = [&](int slot, float m_used, bool held, bool save) {
      float4* sum = reinterpret_cast<float4*>(p.part_o + int64_t(slot) * D);
      const float m_sum = held ? p.part_ml[int64_t(slot) * 2] : -INFINITY;
      const float g = m_sum == -INFINITY ? 0.f : ex2_approx(m_sum - m_used);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tO + c * 32, v);
        tmem_wait_ld();
        reg_fence32(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          if (held) a = sum[c * 8 + i];
          a.x = fmaf(a.x, g, __uint_as_float(v[4 * i]));
          a.y = fmaf(a.y, g, __uint_as_float(v[4 * i + 1]));
          a.z = fmaf(a.z, g, __uint_as_float(v[4 * i + 2]));
          a.w = fmaf(a.w, g, __uint_as_float(v[4 * i + 3]));
          if (save) sum[c * 8 + i] = a;
          v[4 * i] = save ? 0u : __float_as_uint(a.x);
          v[4 * i + 1] = save ? 0u : __float_as_uint(a.y);
          v[4 * i + 2] = save ? 0u : __float_as_uint(a.z);
          v[4 * i + 3] = save ? 0u : __float_as_uint(a.w);
        }
        tmem_st32(tO + c * 32, v);
      }
      tmem_wait_st();
      if (save) p.part_ml[int64_t(slot) * 2] = m_used;
    };
    bool more = take(cur);
    while (more) {
      const RowAt row = cur.row;
      const int nt = cur.nt, slot = cur.slot;
      const bool whole = cur.whole;
      const float qk2 = cur.qk2;
      float m_used = -INFINITY, l_sum = 0.f;
      int seen = cur.seen, held = cur.held, seen_min = cur.seen_min;
      int stop = min(nt, kSumTiles);
      for (int j = 0; j < nt;) {
        for (; j < stop; ++j) {
          ok = wait_all(L::kS + x, s_phase);
          if (!ok) break;
          s_phase ^= 1;
          tc_fence_after();
          float sv[128];
          {
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, v[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              reg_fence32(v[c]);
#pragma unroll
              for (int i = 0; i < 32; ++i) sv[c * 32 + i] = __uint_as_float(v[c][i]);
            }
          }
          if (seen_min < kTileKT) {
#pragma unroll
            for (int c = 0; c < 128; ++c) sv[c] = c < seen ? sv[c] : -INFINITY;
          }
          float m0 = sv[0], m1 = sv[1], m2 = sv[2], m3 = sv[3];
#pragma unroll
          for (int c = 4; c < 124; c += 8) {
            m0 = fmax3(m0, sv[c + 0], sv[c + 1]);
            m1 = fmax3(m1, sv[c + 2], sv[c + 3]);
            m2 = fmax3(m2, sv[c + 4], sv[c + 5]);
            m3 = fmax3(m3, sv[c + 6], sv[c + 7]);
          }
          m0 = fmax3(m0, sv[124], sv[125]);
          m1 = fmax3(m1, sv[126], sv[127]);
          const float m_tile = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * qk2;
          float f = 1.f;
          if (m_tile > m_used + (kRescale + kLift<DT>) || (m_used == -INFINITY && m_tile > -INFINITY)) {
            f = ex2_approx(m_used - (m_tile - kLift<DT>));
            m_used = m_tile - kLift<DT>;
            l_sum *= f;
          }
          if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {   // O_X is stable: S_X(j) came after PV_X(j-1)
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(tO + c * 32, v);
              tmem_wait_ld();
              reg_fence32(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tmem_st32(tO + c * 32, v);
            }
          }
          const float shift = m_used == -INFINITY ? 0.f : -m_used;
#pragma unroll
          for (int c = 0; c < 128; c += 2) ffma2(sv[c], sv[c + 1], sv[c], sv[c + 1], qk2, qk2, shift, shift);
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = ex2_approx(sv[c]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = pack2<DT>(sv[64 * q + 2 * c], sv[64 * q + 2 * c + 1]);
            tmem_st32(tS + q * 32, pk);
          }
          // The values' rows behind the cache's end hold anything, and 0 * NaN
          // must not reach O: tile A's threads clear them (PV_B comes after
          // PV_A, which waits for these threads).
          if (x == 0 && held < kTileKT) {
            ok = wait_all(L::kFull + vr.slot, vr.phase);
            if (!ok) break;
            if (r >= held) {
              const uint32_t dst = sbase + L::kRing + vr.slot * L::kTile + r * 128;
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                st_shared_v4(dst + (c >> 3) * L::kPanel + ((c & 7) << 4), make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_smem();
          }
          vr.skip(2);
          seen -= kTileKT;
          seen_min -= kTileKT;
          held -= kTileKT;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kP + x));
          float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f, a4 = 0.f, a5 = 0.f, a6 = 0.f, a7 = 0.f;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            fadd2(a0, a1, a0, a1, sv[c + 0], sv[c + 1]);
            fadd2(a2, a3, a2, a3, sv[c + 2], sv[c + 3]);
            fadd2(a4, a5, a4, a5, sv[c + 4], sv[c + 5]);
            fadd2(a6, a7, a6, a7, sv[c + 6], sv[c + 7]);
          }
          l_sum += ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
        }
        if (!ok || j == nt) break;
        ok = wait_all(L::kS + x, s_phase);      // O_X is stable then (above waits again)
        if (!ok) break;
        tc_fence_after();
        move_sum(slot, m_used, j > kSumTiles, true);
        stop = min(nt, j + kSumTiles);
      }
      if (!ok) break;
      more = take(cur);
      if (nt > 0) {
        ok = wait_all(L::kO + x, o_phase);
        if (!ok) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      if (__builtin_expect(nt > kSumTiles, 0)) move_sum(slot, m_used, true, false);
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;      // no key: zeros
      auto load_o = [&](int c, uint32_t (&v)[32]) {            // 32 channels of this row
        if (nt > 0) {
          tmem_ld32(tO + c * 32, v);
          tmem_wait_ld();
          reg_fence32(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
      };
      // O by way of the warp's stage, 32 channels of every row at a time: 4 (or,
      // of an fp32 partial, 8) lanes a row, so that global stores are whole
      // sectors.  Loops, not unrolled: code that runs once an item costs most
      // by being fetched.
      const uint32_t stage = sbase + L::kStage + (warp - 4) * L::kStageBytes;
      auto stage_at = [&](int w, int c) { return stage + w * 128 + ((c ^ (w & 7)) << 4); };
      const int lanes_log2 = whole ? 2 : 3;
      const int w0 = lane >> lanes_log2, wc = lane & ((1 << lanes_log2) - 1);
      uint64_t to = 0;
      if (row.token >= 0)
        to = whole ? reinterpret_cast<uint64_t>(p.out + row.token * p.os[0] + row.head * p.os[1])
                   : reinterpret_cast<uint64_t>(p.part_o + int64_t(slot) * D);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        load_o(c, v);
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = pack2<DT>(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < 4 || !whole)
            st_shared_v4(stage_at(lane, i), make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        __syncwarp();
#pragma unroll 1
        for (int it = 0; it < 1 << lanes_log2; it += 4) {
          uint4 o[4];
          uint64_t at[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int w = ((it + q) << (5 - lanes_log2)) + w0;
            at[q] = __shfl_sync(0xffffffffu, to, w);
            o[q] = ld_shared_v4(stage_at(w, wc));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (at[q] != 0) *reinterpret_cast<uint4*>(at[q] + (((c << lanes_log2) + wc) << 4)) = o[q];
        }
        __syncwarp();
      }
      if (row.token >= 0) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + int64_t(slot) * 2) = make_float2(m_used, l_sum);
        else if (p.lse != nullptr)
          p.lse[int64_t(row.token) * p.Hq + row.head] =
              l_sum == 0.f ? -INFINITY : (m_used + log2f(l_sum)) * kLn2;
      }
      tc_fence_before();        // O has been read: the next segment's first PV, after kP, may write it
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ rows kernel
// Few rows a kv head (decoding, drafted tokens): bound by reading the keys and
// values once.  The CTA's items are MT tiles of 16 rows; a loading warp fills a
// ring of 128-key tiles, and 8 warps take 16 keys of every tile each, without a
// barrier among them until an item ends, when their results are added in
// shared memory.  The products run on mma.sync: 16 rows fill its tile where a
// tcgen05 tile would be one eighth full.
//
// Measured (32 heads of 128 over 8 kv heads, bf16): 64 sequences of up to 8190
// rows out of 16-row pages 191 to 206 us with its join, 5.8 to 6.3 TB/s; one of 65536 rows
// 49 us, 5.5 TB/s, of which 7 are finding the share, the handoff and the join.
// 3 to 7 drafted tokens of 24 heads of 64 for each of 32 caches of up to 4000 rows
// 46 us, 3.2 TB/s: 12 us do not shrink with the caches (plan, first loads, items'
// starts and ends, join), and 6 or 7 tokens are two row tiles that read the keys
// twice; each further row costs what 6.2 TB/s take.  Two key tiles at a time in
// a warp: 49 us.  A warp's sum takes an eighth of a share's keys, so what an MMA
// cuts off (see kSumTiles) is 0.1% over 2^20 keys of equal weight.
// (Warps 0-3 are the loader's group; three of them only hand their registers on.)
constexpr int kRowWarps = 8;
constexpr int kRowThreads = kRowWarps * 32 + 128;

template <int DT>
VARK_DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == VARK_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
VARK_DEV void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
VARK_DEV void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int D, int MT>
struct RowSmem {
  static constexpr int kR = 16 * MT;
  static constexpr int kPanel = kTileKT * 128;            // 128 rows x 64 channels
  static constexpr int kTile = (D / 64) * kPanel;         // a tile's keys or values
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kRing = 0;
  static constexpr int kQPanel = kR * 128;
  static constexpr int kQ = kRing + kSlots * kTile;
  static constexpr int kStride = D + 8;                   // floats; + 8 spreads the 8 rows of a store over the banks
  static constexpr int kMerge = kQ + (D / 64) * kQPanel;                         // [warp][16][stride] fp32
  static constexpr int kML = kMerge + kRowWarps * 16 * kStride * 4;             // [warp][16][2] fp32
  static constexpr int kRow = kML + kRowWarps * 16 * 2 * 4;                      // [kR] limit, [kR] scale
  static constexpr int kBar = kRow + kR * 8;
  static constexpr int kFull = 0, kEmpty = kSlots;        // barrier indices
  static constexpr int kMisc = kBar + 2 * kSlots * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc + 2048 <= kMaxSmem, "shared memory");
  // Registers a thread: at launch, then of the loader's group and of the others.
  // What is left of the SM's 65536 lets the join's CTA wait beside this one (two
  // row tiles of 128 channels spill at 200, so there it follows instead).
  static constexpr bool kWide = D * MT > 128;
  static constexpr int kLaunchRegs = kWide ? 168 : 128, kLoadRegs = kWide ? 56 : 48, kWorkRegs = kWide ? 224 : 168;
  static_assert(128 * kLoadRegs + 256 * kWorkRegs <= kRowThreads * kLaunchRegs, "registers");
};

template <int DT, int D, int MT>
__global__ void __launch_bounds__(kRowThreads) __maxnreg__((RowSmem<D, MT>::kLaunchRegs))
rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ AttnParams p) {
  using L = RowSmem<D, MT>;
  using Seg = Segments<L::kR, kTileKT>;
  using Ring = RingAt<L::kSlots>;
  constexpr int KS = D / 16, NT = D / 8, THREADS = kRowWarps * 32;
  constexpr bool kQRegs = MT * KS <= 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* ml = reinterpret_cast<float*>(smem + L::kML);
  int* row_limit = reinterpret_cast<int*>(smem + L::kRow);
  float* row_scale = reinterpret_cast<float*>(smem + L::kRow + L::kR * 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * uint32_t(i); };
  const int warp = int(threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
  const int tid = int(threadIdx.x) - 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bar(L::kFull + i), 1);
      mbar_init(bar(L::kEmpty + i), kRowWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_wait();
  grid_release();           // only now: the join plans before it waits, so what wrote the tables has ended
  const Share share = find_share<L::kR, kTileKT, kRowThreads, false>(p, blockIdx.x);   // syncs the block
  if (share.u0 == share.u1) return;
  if (warp < 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoadRegs) : "memory");
    if (warp == -4) load_tiles<D, L::kR, L>(p, share, tm_k, tm_v, sbase, abort_flag);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kWorkRegs) : "memory");
  auto sync = [&]() { named_bar_sync(1, THREADS); };

  const int g = lane >> 2, t4 = lane & 3;
  // ldmatrix addresses of this lane: a row of a 16 x 16 block, and the 16-byte
  // chunk of each 16-channel step within a panel (128-byte swizzle)
  const int lr = lane & 7, li = lane >> 3;
  uint32_t k_off[4], v_off[4], q_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k_off[i] = (warp * 16 + (li >> 1) * 8 + lr) * 128 + (((i * 2 + (li & 1)) ^ lr) << 4);
    q_off[i] = ((li & 1) * 8 + lr) * 128 + (((i * 2 + (li >> 1)) ^ lr) << 4);
    v_off[i] = warp * 16 * 128 + q_off[i];
  }

  Ring use = {0, 0};
  bool ok = true;
  auto next_slot = [&]() -> uint32_t {      // waits for the next half of a tile
    ok = ok && mbar_wait(bar(L::kFull + use.slot), uint32_t(use.phase), abort_flag, p.status, p.wait_limit_ns);
    ok = __all_sync(0xffffffffu, ok);
    return sbase + L::kRing + use.slot * L::kTile;
  };
  auto release = [&]() {                    // this warp is done with it
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::kEmpty + use.slot));
    use.skip(1);
  };
  // The tile's queries: asked for while the segment before is worked on, then
  // stored 128-byte swizzled with what their rows see and scale by.  Under a
  // negative temperature the query's sign is turned instead, so the largest
  // score gives the largest logit; under 0 the query is 0.
  constexpr int NQ = (L::kR * (D / 8) + THREADS - 1) / THREADS;
  uint4 qw[NQ];
  int q_limit[NQ];
  float q_scale[NQ];
  auto fetch = [&](const Seg& sg) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = (tid + n * THREADS) / (D / 8), ch = tid % (D / 8);
      const RowAt a = row_at(p, sg, r);
      q_limit[n] = a.limit;
      q_scale[n] = p.scale_log2;
      qw[n] = make_uint4(0u, 0u, 0u, 0u);
      if (r < L::kR && a.token >= 0) {
        if (p.tau != nullptr) q_scale[n] *= p.tau[a.head];
        qw[n] = *reinterpret_cast<const uint4*>(p.q + a.token * p.qs[0] + a.head * p.qs[1] + ch * 8);
      }
    }
  };
  auto put = [&]() {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = (tid + n * THREADS) / (D / 8), ch = tid % (D / 8);
      if (r >= L::kR) continue;
      const uint32_t flip = q_scale[n] < 0.f ? 0x80008000u : 0u;
      uint4 w = q_scale[n] == 0.f ? make_uint4(0u, 0u, 0u, 0u) : qw[n];
      w.x ^= flip; w.y ^= flip; w.z ^= flip; w.w ^= flip;
      st_shared_v4(sbase + L::kQ + (ch >> 3) * L::kQPanel + r * 128 + (((ch & 7) ^ (r & 7)) << 4), w);
      if (ch == 0) {
        row_limit[r] = q_limit[n];
        row_scale[r] = q_scale[n] == 0.f ? 1.f : fabsf(q_scale[n]);
      }
    }
  };
  Seg cs, ahead;
  ahead.start(p, share);
  bool more = ahead.next(p);
  if (more) fetch(ahead);
  while (more) {
    put();
    cs = ahead;
    sync();
    more = ahead.next(p);
    if (more) fetch(ahead);
    int lim[MT][2];
    float scale[MT][2], m[MT][2], top[MT][2], l[MT][2], o[MT][NT][4];   // m: the reference; top: the maximum + its lag
    uint32_t qa[kQRegs ? MT * KS : 1][4];   // the A operand, where it fits the registers
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lim[mt][i] = row_limit[mt * 16 + g + 8 * i];
        scale[mt][i] = row_scale[mt * 16 + g + 8 * i];
        m[mt][i] = top[mt][i] = -INFINITY;
        l[mt][i] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][n][i] = 0.f;
    }
    if constexpr (kQRegs) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < KS; ++k)
          ldmatrix4(sbase + L::kQ + mt * 16 * 128 + (k >> 2) * L::kQPanel + q_off[k & 3], qa[mt * KS + k]);
    }
    // keys that every row of the tile sees (the first row sees the fewest)
    const int all_see = cs.tile * L::kR + L::kR <= cs.x.n * p.G ? row_limit[0] : 0;
    const int nt = seen_tiles(p, cs);
    int key0 = cs.k0 * kTileKT + warp * 16;
    for (int j = 0; j < nt; ++j, key0 += kTileKT) {
      const uint32_t sk = next_slot();
      if (!ok) break;
      // two sums a score, over even and odd 16-channel steps: half the chain of
      // dependent MMAs
      float s[MT][2][4], s2[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][n][i] = s2[mt][n][i] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        ldmatrix4(sk + k_off[k & 3] + (k >> 2) * L::kPanel, b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t qf[4];
          if constexpr (kQRegs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) qf[i] = qa[mt * KS + k][i];
          } else {
            ldmatrix4(sbase + L::kQ + mt * 16 * 128 + (k >> 2) * L::kQPanel + q_off[k & 3], qf);
          }
          mma16816<DT>((k & 1) ? s2[mt][0] : s[mt][0], qf, b[0], b[1]);
          mma16816<DT>((k & 1) ? s2[mt][1] : s[mt][1], qf, b[2], b[3]);
        }
      }
      release();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][n][i] += s2[mt][n][i];
      if (key0 + 16 > all_see) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + n * 8 + 2 * t4 + (i & 1) >= lim[mt][i >> 1]) s[mt][n][i] = -INFINITY;
      }
      // Against the running maximum, which may lag by 2^8: the four lanes of a
      // row keep the same one and look for the new one together only when
      // some score has passed it by more.
      float mx[MT][2];
      bool past = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[mt][i] = fmaxf(fmax3(s[mt][0][2 * i], s[mt][0][2 * i + 1], s[mt][1][2 * i]), s[mt][1][2 * i + 1]) *
                      scale[mt][i];
          past |= mx[mt][i] > top[mt][i];
        }
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = fmaxf(mx[mt][i], __shfl_xor_sync(0xffffffffu, mx[mt][i], 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            if (v > top[mt][i]) {
              const float f = ex2_approx(m[mt][i] - (v - kLift<DT>));          // (the first time: 0)
              m[mt][i] = v - kLift<DT>;
              top[mt][i] = v + kRescale;
              l[mt][i] *= f;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                o[mt][n][2 * i] *= f;
                o[mt][n][2 * i + 1] *= f;
              }
            }
          }
      }
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float shift = m[mt][i] == -INFINITY ? 0.f : m[mt][i];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[mt][n][2 * i + e] = ex2_approx(fmaf(s[mt][n][2 * i + e], scale[mt][i], -shift));
          l[mt][i] += (s[mt][0][2 * i] + s[mt][0][2 * i + 1]) + (s[mt][1][2 * i] + s[mt][1][2 * i + 1]);
        }
        // the probabilities, rounded to the values' type, are the A operand of P V
        pa[mt][0] = pack2<DT>(s[mt][0][0], s[mt][0][1]);
        pa[mt][1] = pack2<DT>(s[mt][0][2], s[mt][0][3]);
        pa[mt][2] = pack2<DT>(s[mt][1][0], s[mt][1][1]);
        pa[mt][3] = pack2<DT>(s[mt][1][2], s[mt][1][3]);
      }
      const uint32_t sv = next_slot();
      if (!ok) break;
      // rows behind the cache's end hold anything: 0 * NaN must not reach the sum
      const int left = cs.x.len - key0;
      const bool tail = left < 16;
      const uint32_t keep0 = (2 * t4 < left ? 0xFFFFu : 0u) | (2 * t4 + 1 < left ? 0xFFFF0000u : 0u);
      const uint32_t keep1 = (2 * t4 + 8 < left ? 0xFFFFu : 0u) | (2 * t4 + 9 < left ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        uint32_t b[4];
        ldmatrix4_trans(sv + v_off[c & 3] + (c >> 2) * L::kPanel, b);
        if (tail) {
          b[0] &= keep0;
          b[1] &= keep1;
          b[2] &= keep0;
          b[3] &= keep1;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<DT>(o[mt][2 * c], pa[mt], b[0], b[1]);
          mma16816<DT>(o[mt][2 * c + 1], pa[mt], b[2], b[3]);
        }
      }
      release();
    }
    // the warps' results, each relative to its own maxima, 16 rows at a time
    const bool whole = cs.whole();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 1);
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 2);
        const int r = g + 8 * i;
        float* mo = merge + (warp * 16 + r) * L::kStride + 2 * t4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2*>(mo + n * 8) = make_float2(o[mt][n][2 * i], o[mt][n][2 * i + 1]);
        if (t4 == 0) *reinterpret_cast<float2*>(ml + (warp * 16 + r) * 2) = make_float2(m[mt][i], l[mt][i]);
      }
      sync();
      for (int i = tid; i < 16 * (D / 8); i += THREADS) {
        const int r = i / (D / 8), d0 = (i % (D / 8)) * 8;
        const RowAt a = row_at(p, cs, mt * 16 + r);
        if (a.token < 0 || *abort_flag != 0) continue;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, ml[(w * 16 + r) * 2]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f, acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(ml + (w * 16 + r) * 2);
          const float wgt = ex2_approx(v.x - ref);
          sum = fmaf(v.y, wgt, sum);
          const float* mo = merge + (w * 16 + r) * L::kStride + d0;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(mo[e], wgt, acc[e]);
        }
        if (whole) {
          store_row8<DT>(p, a, d0, acc, top, sum);
        } else {
          const int64_t slot = int64_t(part_slot(blockIdx.x, cs.k0)) * L::kR + mt * 16 + r;
          float4* to = reinterpret_cast<float4*>(p.part_o + slot * D + d0);
          to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
          if (d0 == 0) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(top, sum);
        }
      }
      sync();
    }
  }
}

// Joins partial results.  The CTAs whose shares hold a part of an item share its
// rows, 32 channels at a time: share c takes every n-th of these pieces, n the
// number of parts (dealt on to the gridDim.y CTAs of the share), and finds at
// most two such items, at its two ends: one for each half of its threads.
// Threads that a few pieces would leave idle share the parts of one.  All that
// does not need the partials is done before the attention ends; the CTA waits
// beside a running rows kernel, in the registers that leaves.  Bound by two
// dependent loads after the handoff, 2 to 3 us for few rows, and by reading the
// partials out of L2 for many.  (One CTA per item took 5 us for 19 parts, a row a
// CTA 4; finding the parts again for every piece 1 to 3 more.)
template <int R>
struct JoinShape { static constexpr int kHalf = 128, kSplit = R == kTileR ? 4 : 1; };

template <int DT, int D, int R, int KT>
__global__ void __launch_bounds__(2 * JoinShape<R>::kHalf, 4) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kHalf = JoinShape<R>::kHalf;
  constexpr int kPieces = D / 32;               // of a row
  constexpr int kSlots = kHalf / 4;             // (piece, part) slots of 4 threads, 8 channels each
  __shared__ __align__(16) float red_all[2][kSlots][32 + 4];
  __shared__ float red_ml_all[2][kSlots][2];
  __shared__ int part_all[2][kCtas];            // the first row of a share's part in the workspace, or -1
  __shared__ int whole[2];                      // one share did all of the item
  const int c = blockIdx.x;
  if (threadIdx.x < 2) whole[threadIdx.x] = 0;
  grid_release();
  const Share s = find_share<R, KT, 2 * kHalf, true>(p, c);
  const int k = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
  auto red = red_all[k];
  auto red_ml = red_ml_all[k];
  auto part_row = part_all[k];
  const int d1 = (tid & 3) * 8, slot = tid >> 2;
  Segments<R, KT> seg;
  ItemPlace item = {0, 0, 0};
  int c0 = 0, n = 0;                            // the shares that may hold a part
  bool work = s.u0 != s.u1;
  if (work) work = cut_item(p, s, k, seg);
  if (work) {
    item = seg.at;
    c0 = s.holder(item.from);
    n = s.holder(item.to - 1) - c0 + 1;
    for (int q = tid; q < n; q += kHalf) {       // share c0 + q's part
      int k0, k1;
      part_of<KT>(item, s, c0 + q, k0, k1);
      part_row[q] = k0 < k1 ? part_slot(c0 + q, k0) * R : -1;
      if (k0 == 0 && k1 == item.key_tiles) whole[k] = 1;
    }
  }
  __syncthreads();
  work = work && !whole[k];
  const int pieces = work ? min(R, seg.x.n * p.G - seg.tile * R) * kPieces : 0;
  const int first = c - c0 + int(blockIdx.y) * n, step = n * int(gridDim.y);
  const int mine = work ? (pieces - first + step - 1) / step : 0;
  // Every CTA waits, also those without an item: the launch after this one
  // may count on the attention kernel's end.
  grid_wait();
  if (mine <= 0) return;
  const int32_t status = *reinterpret_cast<volatile int32_t*>(p.status);
  for (int r0 = 0; r0 < mine; r0 += kSlots) {
    int width = 1;                              // slots of a part
    while (width < min(kSlots, mine - r0)) width *= 2;
    const int parts = kSlots / width;
    const int i0 = r0 + slot % width, piece = first + i0 * step;
    const int r = piece / kPieces, d0 = piece % kPieces * 32 + d1;
    float top = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    if (i0 < mine) {
      constexpr int kBatch = 2;                 // partials in flight a thread
      for (int q0 = slot / width; q0 < n; q0 += kBatch * parts) {
        float2 v[kBatch];
        float4 w[kBatch][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int q = q0 + b * parts;
          v[b] = make_float2(-INFINITY, 0.f);
          w[b][0] = w[b][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          const int row = q < n ? part_row[q] : -1;
          if (row >= 0) {
            const int64_t from = row + r;
            v[b] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + from * 2));
            w[b][0] = __ldcg(reinterpret_cast<const float4*>(p.part_o + from * D + d0));
            w[b][1] = __ldcg(reinterpret_cast<const float4*>(p.part_o + from * D + d0 + 4));
          }
        }
        float big = top;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) big = fmaxf(big, v[b].x);
        const float ref = big == -INFINITY ? 0.f : big;
        const float old = ex2_approx(top - ref);
        top = big;
        sum *= old;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const float wgt = ex2_approx(v[b].x - ref);
          sum = fmaf(v[b].y, wgt, sum);
          const float z[8] = {w[b][0].x, w[b][0].y, w[b][0].z, w[b][0].w,
                              w[b][1].x, w[b][1].y, w[b][1].z, w[b][1].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(z[e], wgt, acc[e]);
        }
      }
    }
    if (parts > 1) {
      named_bar_sync(1 + k, kHalf);
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&red[slot][d1 + e]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      if (d1 == 0) {
        red_ml[slot][0] = top;
        red_ml[slot][1] = sum;
      }
      named_bar_sync(1 + k, kHalf);
      if (slot < width) {
        float big = top;
        for (int q = 1; q < parts; ++q) big = fmaxf(big, red_ml[slot + q * width][0]);
        const float ref = big == -INFINITY ? 0.f : big;
        const float own = ex2_approx(top - ref);
        top = big;
        sum *= own;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= own;
#pragma unroll 4
        for (int q = 1; q < parts; ++q) {
          const float wgt = ex2_approx(red_ml[slot + q * width][0] - ref);
          sum = fmaf(red_ml[slot + q * width][1], wgt, sum);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(red[slot + q * width][d1 + e], wgt, acc[e]);
        }
      }
    }
    if (slot < width && i0 < mine && status == 0) store_row8<DT>(p, row_at(p, seg, r), d0, acc, top, sum);
  }
}

// ------------------------------------------------------------------ host side
// Rows of an item, from the call's shapes alone (the lengths are on the
// device): the mean rows a (sequence, kv head) decide.  Up to 16 one row tile
// (16 rows over 2 x 20000 keys, D = 128: 27 us against 30 as two tiles and 43
// on tcgen05); up to 32 two (20 rows: 31, 33 as one at a time, 42); D = 64 two
// at a time up to 64 (64 rows: 32 against 35 on tcgen05, 96: 41 against 34);
// beyond that 256 on tcgen05 (D = 128, 48 rows: 43 against 45; 96: 44 against 59).
// All of these were batches of sequences with about as many tokens each.  A chunk
// among sequences that decode goes the mean's way, which is slow for it: 255 of
// one token and one of 1700 over caches of 3000 rows 1059 us in one call, 618 as
// two; 63 and one of 2048 293 and 290.
static int choose_rows(int64_t n_tokens, int B, int Hq, int Hkv, int D) {
  const int64_t rows = n_tokens * (Hq / Hkv);         // of a kv head, over all sequences
  return rows <= int64_t(B) * 16 ? 16 : rows <= int64_t(B) * (D == 64 ? 64 : 32) ? 32 : kTileR;
}

static void test_hooks(AttnParams& p) {
  p.wait_limit_ns = kWaitLimitNs;
  p.withhold = -1;
  if (const char* e = std::getenv("VARK_TEST_WAIT_LIMIT_MS")) {
    const long ms = std::strtol(e, nullptr, 10);
    if (ms > 0 && ms <= 10000) p.wait_limit_ns = uint64_t(ms) * 1000000ull;
  }
  if (const char* e = std::getenv("VARK_TEST_WITHHOLD_KV_TILE")) {
    const long j = std::strtol(e, nullptr, 10);
    if (j >= 0 && j < (1 << 20)) p.withhold = int(j);
  }
}

static int encode_pages(CUtensorMap* m, const uint16_t* base, const Pages& pg, int D, int box_rows) {
  const uint64_t rows = uint64_t(pg.page_heads) << pg.log2_page;
  const uint64_t dims[3] = {uint64_t(D), rows, uint64_t(pg.n_pages)};
  const uint64_t strides[2] = {uint64_t(D) * 2, rows * D * 2};
  return encode_bf16_map(m, base, 3, dims, strides, uint32_t(box_rows));   // 16-bit elements, copied as they are
}

// Lets a kernel use more than 48 KB of shared memory; asked for once a device.
template <typename K>
static int allow_smem(K kern, int smem, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VARK_E_CUDA;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done->load(std::memory_order_relaxed) & bit) return VARK_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return VARK_E_CUDA;
  }
  if (dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return VARK_OK;
}

template <int DT, int D>
static int launch_tiles(const CUtensorMap& k, const CUtensorMap& v, const AttnParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = TileSmem<D>::kAlloc;
  int rc = allow_smem(tiles_kernel<DT, D>, smem, &done);
  if (!rc) rc = launch_early(tiles_kernel<DT, D>, dim3(kCtas), kTileThreads, smem, st, k, v, p);
  if (rc) return rc;
  using J = JoinShape<kTileR>;
  return launch_early(join_kernel<DT, D, kTileR, kTileKT>, dim3(kCtas, J::kSplit), 2 * J::kHalf, 0, st, p);
}

template <int DT, int D, int MT>
static int launch_rows(const CUtensorMap& k, const CUtensorMap& v, const AttnParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = RowSmem<D, MT>::kAlloc;
  int rc = allow_smem(rows_kernel<DT, D, MT>, smem, &done);
  if (!rc) rc = launch_early(rows_kernel<DT, D, MT>, dim3(kCtas), kRowThreads, smem, st, k, v, p);
  if (rc) return rc;
  return launch_early(join_kernel<DT, D, 16 * MT, kTileKT>, dim3(kCtas), 2 * JoinShape<16 * MT>::kHalf, 0, st, p);
}

template <int DT>
static int launch(int D, int rows, const CUtensorMap& k, const CUtensorMap& v, const AttnParams& p, cudaStream_t st) {
  if (rows == kTileR) return D == 128 ? launch_tiles<DT, 128>(k, v, p, st) : launch_tiles<DT, 64>(k, v, p, st);
  if (rows == 32) return D == 128 ? launch_rows<DT, 128, 2>(k, v, p, st) : launch_rows<DT, 64, 2>(k, v, p, st);
  return D == 128 ? launch_rows<DT, 128, 1>(k, v, p, st) : launch_rows<DT, 64, 1>(k, v, p, st);
}

// Rows of the call are counted in 30 bits, entries of the length table in 24.
static int check_shapes(int64_t n_tokens, int B, int Hq, int Hkv, int D) {
  if (D != 64 && D != 128) return VARK_E_SHAPE;
  if (n_tokens < 0 || B < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65536) return VARK_E_SHAPE;
  if (n_tokens > INT32_MAX / 2 / Hq || int64_t(B) * Hkv > (1 << 24)) return VARK_E_SHAPE;
  return VARK_OK;
}

// The plan's units (see Entry) add up in 64 bits whatever the tables hold:
// offsets that go up and down give at most every other sequence all tokens
// (recorded, but by then they are summed).
static bool plan_fits(int64_t n_tokens, int B, int Hq, int Hkv, int64_t max_rows) {
  const double row_tiles = double((int64_t(B) + 1) / 2) * (double(n_tokens) * Hq / 16 + Hkv);
  const double heaviest = kUnit * (double(max_rows) + double(n_tokens) + 512);
  return row_tiles * heaviest < 4.6e18;
}

static int64_t workspace_bytes_for(int rows, int D) { return int64_t(kCtas) * 2 * rows * (D + 2) * 4; }

}  // namespace paged
}  // namespace vark

using namespace vark;
using namespace vark::paged;

extern "C" int64_t vark_paged_attention_workspace(int64_t n_tokens, int B, int Hq, int Hkv, int D, int page_size,
                                                  int max_pages) {
  if (const int rc = check_shapes(n_tokens, B, Hq, Hkv, D)) return rc;
  if (page_size < 1 || max_pages < 1) return VARK_E_SHAPE;
  return workspace_bytes_for(choose_rows(n_tokens, 1, Hq, Hkv, D), D);      // (fewer sequences: as many rows or more)
}

extern "C" int vark_paged_attention(int dtype, const uint16_t* q, const int64_t* q_strides, int64_t n_tokens, int B,
                                    int Hq, int Hkv, int D, const int32_t* cu_tokens, const uint16_t* k_pages,
                                    const uint16_t* v_pages, int64_t n_pages, int page_size,
                                    const int32_t* page_table, int max_pages, const int32_t* cache_len,
                                    int head_pages, const float* tau, int causal, uint16_t* out,
                                    const int64_t* out_strides, float* lse, void* workspace, int64_t workspace_bytes,
                                    int32_t* dev_status, void* stream) {
  if (!dev_status || (dtype != VARK_BF16 && dtype != VARK_FP16)) return VARK_E_ARG;
  int rc = check_shapes(n_tokens, B, Hq, Hkv, D);
  if (rc) return rc;
  AttnParams p;
  if ((rc = make_pages(&p.pg, page_table, cache_len, n_pages, page_size, max_pages, Hkv, head_pages))) return rc;
  if (!plan_fits(n_tokens, B, Hq, Hkv, int64_t(max_pages) * page_size)) return VARK_E_SHAPE;
  if (n_tokens == 0 || B == 0) return check_device_sm100();       // empty tensors have no addresses to look at
  if (!q || !q_strides || !cu_tokens || !k_pages || !v_pages || !page_table || !cache_len || !out || !out_strides ||
      !workspace)
    return VARK_E_ARG;
  const int rows = choose_rows(n_tokens, B, Hq, Hkv, D);
  if (workspace_bytes < workspace_bytes_for(rows, D)) return VARK_E_ARG;
  const int64_t extent[2] = {n_tokens, Hq};
  if (!take_strides(p.qs, q_strides, extent, 2, 0) || !take_strides(p.os, out_strides, extent, 2, D))
    return VARK_E_ALIGN;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned16(workspace))
    return VARK_E_ALIGN;
  if ((rc = check_device_sm100())) return rc;
  p.q = q; p.out = out; p.lse = lse;
  p.cu = cu_tokens;
  p.tau = tau;
  p.N = n_tokens;
  p.B = B; p.G = Hq / Hkv; p.Hq = Hq; p.causal = causal != 0;
  p.by_group = FastDiv::of(p.G);
  p.by_heads = FastDiv::of(Hkv);
  p.scale_log2 = kLog2e / sqrtf(float(D));
  p.tokens_per_tile = rows / p.G;
  p.tile_step = rows * kUnit / p.G;
  p.part_ml = static_cast<float*>(workspace);
  p.part_o = p.part_ml + int64_t(kCtas) * 2 * rows * 2;
  p.status = dev_status;
  test_hooks(p);
  const int box = page_size < kTileKT ? page_size : kTileKT;
  CUtensorMap tk, tv;
  if ((rc = encode_pages(&tk, k_pages, p.pg, D, box))) return rc;
  if ((rc = encode_pages(&tv, v_pages, p.pg, D, box))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == VARK_BF16 ? launch<VARK_BF16>(D, rows, tk, tv, p, st) : launch<VARK_FP16>(D, rows, tk, tv, p, st);
}
