// Shared by the paged-cache operators: 16-bit element types, the row
// arithmetic of a paged pool, and the sequence tables of a ragged batch.
#pragma once

#include "vark_common.cuh"

namespace vark {
namespace paged {

// Records the first error of a call in the caller's status word.
VARK_DEV void record(int32_t* status, int32_t code) { atomicCAS(status, 0, code); }

// Dependent launches.  A call's kernels, and calls that follow one another,
// overlap at their ends: a kernel lets the next one start early, and the next
// one waits for it (and all before it) before it touches what it may have
// written.
VARK_DEV void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
VARK_DEV void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch that may start before the kernels ahead of it have ended (see
// grid_wait).
template <typename K, typename... A>
inline int launch_early(K kern, dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return VARK_OK;
  cudaGetLastError();
  return VARK_E_CUDA;
}

// Two 16-bit values of element type DT (VARK_BF16, VARK_FP16) to and from fp32.
template <int DT>
VARK_DEV void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (DT == VARK_BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
  }
}
template <int DT>
VARK_DEV uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (DT == VARK_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

VARK_DEV uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The pages of one call.  A pool is [n_pages][page_heads][page_size][D]; the
// table is [B][table_heads][max_pages] and the lengths [B][table_heads], with
// (page_heads, table_heads) = (H, 1), or (1, H) for head-specific pages.
struct Pages {
  const int32_t* table;
  const int32_t* len;
  int64_t n_pages;
  int max_pages;
  int log2_page;
  int heads;           // kv heads H
  int page_heads;
  int table_heads;
};

// Strides of rows of 16-byte vectors (host): multiples of 8 elements, at least
// `least` (0 for rows that are read, D for rows that are written); the stride of
// an axis of one entry is not looked at.
inline bool take_strides(int64_t* to, const int64_t* s, const int64_t* extent, int n, int least) {
  for (int i = 0; i < n; ++i) {
    to[i] = extent[i] > 1 ? s[i] : 0;
    if (extent[i] > 1 && (s[i] < least || s[i] % 8 != 0)) return false;
  }
  return true;
}

// No two written rows share an element (host, strides as taken above): from the
// smallest stride on, every axis steps over all that the ones before it span.
inline bool rows_apart(const int64_t* s, const int64_t* extent, int n, int D) {
  int64_t span = D, below = 0;
  for (int k = 0; k < n; ++k) {           // the k-th smallest stride, of few
    int at = -1;
    for (int i = 0; i < n; ++i)
      if (extent[i] > 1 && s[i] > below && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) break;
    int alike = 0;                        // two axes of one stride lie on each other
    for (int i = 0; i < n; ++i) alike += extent[i] > 1 && s[i] == s[at];
    if (alike > 1 || s[at] < span) return false;
    below = s[at];
    span = s[at] > (INT64_MAX - span) / extent[at] ? INT64_MAX : span + s[at] * (extent[at] - 1);
  }
  return true;
}

// Checks and fills the page geometry (host).
inline int make_pages(Pages* p, const int32_t* table, const int32_t* len, int64_t n_pages, int page_size,
                      int max_pages, int H, int head_pages) {
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return VARK_E_SHAPE;
  if (n_pages < 1 || n_pages > INT32_MAX || max_pages < 1) return VARK_E_SHAPE;
  if (int64_t(max_pages) * page_size > INT32_MAX - 1024) return VARK_E_SHAPE;   // key indices, and a tile past them
  p->table = table;
  p->len = len;
  p->n_pages = n_pages;
  p->max_pages = max_pages;
  p->log2_page = 0;
  while ((1 << p->log2_page) < page_size) ++p->log2_page;
  p->heads = H;
  p->page_heads = head_pages ? 1 : H;
  p->table_heads = head_pages ? H : 1;
  return VARK_OK;
}

}  // namespace paged
}  // namespace vark
