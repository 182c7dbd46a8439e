// The paged key/value cache as the kernels see it. Internal header.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sa_common.cuh"

namespace sa {

inline int dtype_bytes(int dtype) { return dtype == SA_DTYPE_E4M3 ? 1 : dtype == SA_DTYPE_FP32 ? 4 : 2; }

// Location codes of the status word.
enum { kWherePagedLen = 700, kWherePagedPage = 701, kWherePagedRange = 702 };

// Quotient by a fixed divisor for 0 <= n < 2^31: (mulhi(m, n) + n) >> sh, by
// Granlund and Montgomery's method for invariant divisors (1994); n's bound keeps
// the sum within 32 bits.
struct Divisor {
  uint32_t m = 1;
  int sh = 0;
  Divisor() = default;
  explicit Divisor(uint32_t p) {
    while ((1ull << sh) < p) ++sh;
    m = (uint32_t)((((1ull << sh) - p) << 32) / p + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> sh);
  }
};

struct PagedView {
  char* k;
  char* v;
  const int32_t* table;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  int64_t sp, sh, ss;  // byte strides: page, head, slot
  int64_t table_stride;
  int n_seq, hkv, page_size, n_pages, capacity;
  Divisor by_page;  // quotients by page_size
  // page and slot strides in units of the largest power of two (bytes) that
  // divides both: every row's offset is below 2^32 units (checked on the host)
  uint32_t unit, sp_units, ss_units;
};

// Largest power of two that divides both strides (bytes), and whether a pool's
// last row starts below 2^32 of it.
inline uint32_t paged_unit(int64_t sp, int64_t ss) {
  const int64_t both = sp | ss;
  return both == 0 || (both & 0xffff) == 0 ? 1u << 16 : (uint32_t)(both & -both);
}
inline bool paged_span_ok(const sa_paged_cache& c, int64_t e) {
  const int64_t sp = c.strides[0] * e, ss = c.strides[2] * e, u = paged_unit(sp, ss);
  return (double)sp / u * (c.n_pages - 1) + (double)ss / u * (c.page_size - 1) < 4294967295.0;
}


// Positions of the longest sequence.
inline int paged_capacity(const sa_paged_cache& c) {
  return c.max_len ? c.max_len : c.max_pages * c.page_size;
}

inline PagedView make_paged_view(const sa_paged_cache& c) {
  PagedView p{};
  const int64_t e = dtype_bytes(c.dtype);
  p.k = (char*)c.k;
  p.v = (char*)c.v;
  p.table = c.page_table;
  p.lens = c.seq_lens;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.sp = c.strides[0] * e;
  p.sh = c.strides[1] * e;
  p.ss = c.strides[2] * e;
  p.table_stride = c.table_stride;
  p.n_seq = c.n_seq;
  p.hkv = c.num_kv_heads;
  p.page_size = c.page_size;
  p.by_page = Divisor((uint32_t)c.page_size);
  p.unit = paged_unit(p.sp, p.ss);
  p.sp_units = (uint32_t)(p.sp / p.unit);
  p.ss_units = (uint32_t)(p.ss / p.unit);
  p.n_pages = c.n_pages;
  p.capacity = paged_capacity(c);
  return p;
}

// A sequence's length, inside 0 .. capacity; *bad is set where it was not.
__device__ __forceinline__ int paged_len(const PagedView& p, int s, bool* bad) {
  const int n = p.lens[s];
  const int m = min(max(n, 0), p.capacity);
  if (m != n) *bad = true;
  return m;
}

// Byte offset of position `pos` (below the capacity) in a pool, head 0, by the
// given table row; -1 where the page is not one of the pool's.
__device__ __forceinline__ int64_t paged_row(const PagedView& p, const int32_t* row, int pos) {
  const int i = p.by_page(pos);
  const int page = row[i];
  if ((unsigned)page >= (unsigned)p.n_pages) return -1;
  return page * p.sp + (int64_t)(pos - i * p.page_size) * p.ss;
}

// The positions a query at length n sees: [0, first) and [lo, n); `count` of them.
struct Visible {
  int first, lo, count;
  __device__ Visible(int n, int window, int sinks) {
    lo = window > 0 ? max(0, n - window) : 0;
    first = min(sinks, lo);
    count = first + n - lo;
  }
  __device__ int pos(int c) const { return c < first ? c : c - first + lo; }
};

// A paged operator's kernels are launched so that their blocks may be resident
// before the stream's previous kernel has ended (its last microseconds hide the
// launch). Each touches nothing that a kernel may have written, or may read,
// before all earlier ones have completed, and then lets the next one start.
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_earlier_kernels() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, int cluster, const A&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sa
