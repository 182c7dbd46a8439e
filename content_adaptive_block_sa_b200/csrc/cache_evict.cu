// Eviction from a paged cache by accumulated weight.
//
// For each (sequence, key/value head): the first `sinks`, the last `recent` and
// the positions of the highest weights between them, `budget` in all, move to
// the front in ascending order. The bound is memory: every weight is read once,
// every kept row read and written once.
//
// Selection: one block of 1024 threads per row (a cluster of them where a few rows
// may be above 32K) keeps the row's weights in shared memory as order-preserving 32-bit
// keys and finds the r-th largest by a radix select of 11, 11 and 10 bits, then
// writes the kept positions in order. Shared-memory atomics count 32 keys a
// cycle however close together they lie, so the passes cost their barriers, not
// their keys. The blocks of a cluster read each other's histograms and counts
// through distributed shared memory.
//
// Movement, a second launch: to other pages, a warp takes 32 rows (a lane looks
// up one, the warp copies them two to eight at a time); in place, a block takes
// a slice of the columns (a part of the keys' or values' bytes, or the scores)
// of one (sequence, head) and moves its rows tile by tile. Kept row i comes from
// a position >= i, so a tile that is read before it is written overwrites
// nothing that a later tile still has to read.
//
// Measured: 16 sequences of 20000..32768 to 8192, 8 heads of 128 bf16: 190 us, of
// them 167 the movement at the rate of a copy and 22 the selection; one sequence
// of 8192 to 2048: 13 us, the selection's barriers and the chain position -> page
// -> row; 48 e4m3 sequences of 700..16000 to 1000: 29 us.
// In place, where one block moves a slice of a row's columns in order: 408, 22, 36.
#include <cooperative_groups.h>
#include <math.h>

#include "paged.cuh"

namespace sa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCachedKeys = 32768;  // keys of a block that shared memory holds
constexpr int kMoveThreads = 256;
constexpr int kSms = 148;
// counts[s]: kept positions, and what the movement has to know of the sequence
constexpr int kCountMask = 0x7fffffff, kBadLen = ~kCountMask;

struct EvictArgs {
  PagedView c;
  const float* scores_in;
  float* scores_out;
  const int32_t* dst_table;
  int64_t dst_stride;
  int32_t* keep;
  int32_t* lens_out;
  int32_t* counts;
  DeviceStatus* status;
  int64_t ss, sh, os, oh;
  int budget, sinks, recent, row_bytes;
  int cluster;       // blocks of a row's selection
  int held;          // keys that one of them holds, in rounds of its warps' tiles
  int most;          // positions that a row can keep
  int pieces;        // in place: column slices of keys and of values; 0: other pages
  int scores_apart;  // scores_out is another array
};

// Order-preserving key of a weight: NaN is taken for -inf, -0 for 0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One position written where the comparison holds: a predicated instruction, since
// a branch for each key costs more than the stores that it saves.
__device__ __forceinline__ void store_if_above(uint32_t a, uint32_t b, int32_t* to, int v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.gt.u32 p, %0, %1;\n\t@p st.global.u32 [%2], %3;\n\t}" ::"r"(a),
               "r"(b), "l"(to), "r"(v)
               : "memory");
}

struct SelectShared {
  uint32_t hist[2][kBins];
  uint32_t sums[kSelWarps], found_bin, found_left, found_count, counts[2];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
};

// Keeps the best `left` of the weights w[a.sinks .. end) of a row that C blocks
// share. kHold: shared memory holds the block's keys; else every pass reads the
// weights. The passes stay a loop: a row's few microseconds are bound by the
// fetching of instructions that run once.
template <bool kHold>
__device__ __forceinline__ void select_row(const EvictArgs& a, SelectShared& sh, uint32_t* cached,
                                           const float* w, int32_t* keep, int end, uint32_t left, int C,
                                           int rank) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto& hist = sh.hist;
  auto& sums = sh.sums;
  auto& warp_gt = sh.warp_gt;
  auto& warp_eq = sh.warp_eq;
  auto& counts = sh.counts;
  auto sync_row = [&]() {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  // this warp's share of the row, in order over ranks and warps: tiles of 128
  // keys, four neighbours a lane; 0, below every weight, stands behind the end
  const int tiles = (end - a.sinks + C * kSelWarps * 128 - 1) / (C * kSelWarps * 128);
  const int j0 = a.sinks + (rank * kSelWarps + warp) * tiles * 128;
  uint32_t* mine = cached + warp * tiles * 128;
  auto keys_at = [&](int i) {  // of tile i
    if (kHold) return *(const uint4*)(mine + i * 128 + lane * 4);
    const int j = j0 + i * 128 + lane * 4;
    return make_uint4(j < end ? weight_key(w[j]) : 0, j + 1 < end ? weight_key(w[j + 1]) : 0,
                      j + 2 < end ? weight_key(w[j + 2]) : 0, j + 3 < end ? weight_key(w[j + 3]) : 0);
  };

  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
    uint32_t* h = hist[pass & 1];
    for (int i = tid; i < bins; i += kSelThreads) h[i] = 0;
    __syncthreads();
    if (pass == 0 && kHold) {
#pragma unroll 8
      for (int i = lane; i < tiles * 128; i += 32) {
        const uint32_t key = j0 + i < end ? weight_key(w[j0 + i]) : 0;
        mine[i] = key;
        atomicAdd(&h[key >> 21], 1);
      }
      __syncwarp();
    } else {
      const int known = pass == 0 ? 32 : shift + (pass == 2 ? 10 : 11);  // the bits above are the prefix's
      auto count = [&](uint32_t key) {
        if (known == 32 || key >> known == prefix) atomicAdd(&h[(key >> shift) & (bins - 1)], 1);
      };
#pragma unroll 2
      for (int i = 0; i < tiles; ++i) {
        const uint4 k = keys_at(i);
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      }
    }
    sync_row();
    // the bin that holds the left-th largest key: sums from the top, two bins a
    // thread (half of the threads in the last pass)
    uint32_t c0 = 0, c1 = 0;
    const int b0 = bins - 2 - tid * 2;
    if (b0 >= 0) {
      for (int r = 0; r < C; ++r) {
        const uint2 x = *(const uint2*)((C > 1 ? cluster.map_shared_rank(h, r) : h) + b0);
        c0 += x.y;
        c1 += x.x;
      }
    }
    const uint32_t total = c0 + c1;
    uint32_t upto = total;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, upto, i);
      if (lane >= i) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    const uint32_t above = upto - total + __reduce_add_sync(~0u, lane < warp ? sums[lane] : 0);
    if (above < left && left <= above + total) {
      const bool second = left > above + c0;
      sh.found_bin = b0 + (second ? 0 : 1);
      sh.found_left = left - above - (second ? c0 : 0);
      sh.found_count = second ? c1 : c0;
    }
    __syncthreads();
    prefix = prefix << (pass == 2 ? 10 : 11) | sh.found_bin;
    left = sh.found_left;
    if (left == sh.found_count) {  // the whole bin is kept: the lower bits do not matter
      prefix = (prefix << shift) - 1;
      left = 0;
      break;
    }
  }

  // keys above `prefix` are kept, and the first `left` that equal it
  uint32_t gt = 0, eq = 0;
#pragma unroll 2
  for (int i = 0; i < tiles; ++i) {
    const uint4 k = keys_at(i);
    gt += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
    eq += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
  }
  gt = __reduce_add_sync(~0u, gt);
  eq = __reduce_add_sync(~0u, eq);
  if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
  __syncthreads();
  if (C > 1) {
    if (warp < 2) {
      const uint32_t x = __reduce_add_sync(~0u, (warp ? warp_eq : warp_gt)[lane]);
      if (lane == 0) counts[warp] = x;
    }
    cluster.sync();
  }
  uint32_t ng = 0, ne = 0;
  for (int r = 0; r < rank; ++r) {
    const uint32_t* x = cluster.map_shared_rank(counts, r);
    ng += x[0];
    ne += x[1];
  }
  ng += __reduce_add_sync(~0u, lane < warp ? warp_gt[lane] : 0);
  ne += __reduce_add_sync(~0u, lane < warp ? warp_eq[lane] : 0);
  int32_t* to = keep + a.sinks;
  auto upto_lane = [&](uint32_t x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
#pragma unroll 1
  for (int i = 0; i < tiles; i += 4) {
    // four tiles at once: a byte of `own` counts the lane's keys of a tile
    uint4 k[4];
    uint32_t own = 0;
    bool ties = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      k[u] = make_uint4(0, 0, 0, 0);
      if (i + u >= tiles) continue;
      k[u] = keys_at(i + u);
      own |= (uint32_t)((k[u].x > prefix) + (k[u].y > prefix) + (k[u].z > prefix) + (k[u].w > prefix))
             << (8 * u);
      ties |= k[u].x == prefix || k[u].y == prefix || k[u].z == prefix || k[u].w == prefix;
    }
    if (!__any_sync(~0u, ties && ne < left)) {  // keys that equal it are left out here, or absent
      const uint32_t upto = upto_lane(own), all = __shfl_sync(~0u, upto, 31);
      const uint32_t before = upto - own;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i + u >= tiles) break;
        uint32_t at = ng + min(ne, left) + (before >> (8 * u) & 0xff);
        const int j = j0 + (i + u) * 128 + lane * 4;
        store_if_above(k[u].x, prefix, to + at, j);
        at += k[u].x > prefix;
        store_if_above(k[u].y, prefix, to + at, j + 1);
        at += k[u].y > prefix;
        store_if_above(k[u].z, prefix, to + at, j + 2);
        at += k[u].z > prefix;
        store_if_above(k[u].w, prefix, to + at, j + 3);
        ng += all >> (8 * u) & 0xff;
      }
      continue;
    }
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
      const uint4 k4 = u == 0 ? k[0] : u == 1 ? k[1] : u == 2 ? k[2] : k[3];
      const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
      const int j = j0 + (i + u) * 128 + lane * 4;
      uint32_t g4 = 0, e4 = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) g4 += key[x] > prefix, e4 += key[x] == prefix;
      const uint32_t both = g4 | e4 << 16, upto = upto_lane(both);
      uint32_t pg = ng + ((upto - both) & 0xffff), pe = ne + ((upto - both) >> 16);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (key[x] > prefix) {
          to[pg++ + min(pe, left)] = j + x;
        } else if (key[x] == prefix) {
          if (pe < left) to[pg + pe] = j + x;
          ++pe;
        }
      }
      const uint32_t all = __shfl_sync(~0u, upto, 31);
      ng += all & 0xffff;
      ne += all >> 16;
    }
  }
  if (C > 1) cluster.sync();  // the counts stay until every block has read them
}

// kAll: the block's shared memory (a.held keys) holds its part of every row, or
// else of those that are short enough. Two blocks an SM, though a few registers
// spill: 192 rows on 148 SMs measured 28.7 us a call, with one block an SM 30.9.
template <bool kAll>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t cached[];
  __shared__ __align__(16) SelectShared sh;
  wait_for_earlier_kernels();
  let_next_kernel_start();
  int C = a.cluster;
  const int rank = C > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / C;
  const int s = (int)(row / a.c.hkv), g = (int)(row % a.c.hkv);
  bool bad = false;
  const int len = paged_len(a.c, s, &bad);
  const int n = min(len, a.budget);
  int32_t* keep = a.keep + row * a.budget;
  if (blockIdx.x == 0 && tid == 0) a.status->code = a.status->where = 0;
  if (g == 0 && rank == 0 && tid == 0) a.counts[s] = n | (bad ? kBadLen : 0);
  const int t0 = rank * kSelThreads + tid, step = C * kSelThreads;
  if (len <= a.budget) {
    for (int i = t0; i < a.budget; i += step) keep[i] = i < len ? i : -1;
    return;
  }
  const int end = len - a.recent;
  if (C > 1 && end - a.sinks <= a.held) {  // one block of the cluster does
    if (rank > 0) return;
    C = 1;
  }
  for (int i = rank * kSelThreads + tid; i < a.sinks; i += C * kSelThreads) keep[i] = i;
  for (int i = rank * kSelThreads + tid; i < a.recent; i += C * kSelThreads)
    keep[a.budget - a.recent + i] = end + i;
  const uint32_t left = a.budget - a.sinks - a.recent;
  if (left == 0) return;
  const float* w = a.scores_in + s * a.ss + g * a.sh;
  if (kAll || (end - a.sinks + C - 1) / C <= a.held)
    select_row<true>(a, sh, cached, w, keep, end, left, C, rank);
  else
    select_row<false>(a, sh, cached, w, keep, end, left, C, rank);
}

// In place: the rows of one (sequence, head), `vecs` 16-byte columns from `base`.
__device__ void move_columns(const EvictArgs& a, int s, int g, char* base, int vecs, int n) {
  constexpr int U = 8;
  const int32_t* keep = a.keep + ((int64_t)s * a.c.hkv + g) * a.budget;
  const int32_t* table = a.c.table + s * a.c.table_stride;
  const int vec = threadIdx.x % vecs, r = threadIdx.x / vecs, per = kMoveThreads / vecs;
  char* const column = base + g * a.c.sh + vec * 16;
  const int tile = per * U;
  int64_t from[U];
  uint4 x[U];
  auto look_up = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * per + r;
      from[u] = i < n ? paged_row(a.c, table, keep[i]) : -1;
    }
  };
  look_up(0);
  for (int i0 = 0; i0 < n; i0 += tile) {
    int64_t was[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      was[u] = from[u];
      if (was[u] >= 0) x[u] = *(const uint4*)(column + was[u]);
    }
    look_up(i0 + tile);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * per + r;
      if (i >= n) continue;
      const int64_t at = paged_row(a.c, table, i);
      if (was[u] < 0 || at < 0) {
        if (vec == 0) report(a.status, SA_ERR_DEVICE, kWherePagedPage);
      } else if (at != was[u]) {
        *(uint4*)(column + at) = x[u];
      }
    }
  }
}

// In place: the scores of one (sequence, head).
__device__ void move_scores(const EvictArgs& a, int s, int g, int n) {
  constexpr int U = 8;
  const int32_t* keep = a.keep + ((int64_t)s * a.c.hkv + g) * a.budget;
  float* w = a.scores_out + s * a.os + g * a.oh;
  for (int i0 = 0; i0 < n; i0 += kMoveThreads * U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads + threadIdx.x;
      x[u] = i < n ? w[keep[i]] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads + threadIdx.x;
      if (i < n) w[i] = x[u];
    }
  }
}

// What either movement does for its sequence beside the rows, once.
__device__ __forceinline__ void finish_sequence(const EvictArgs& a, int s, int count) {
  a.lens_out[s] = count & kCountMask;
  if (count & kBadLen) report(a.status, SA_ERR_DEVICE, kWherePagedLen);
}

// Grid: (slice of the columns, head, sequence).
__global__ void __launch_bounds__(kMoveThreads)
    evict_in_place_kernel(const __grid_constant__ EvictArgs a) {
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const int slice = blockIdx.x, g = blockIdx.y, s = blockIdx.z;
  const int count = a.counts[s], n = count & kCountMask;
  if (slice == 0 && g == 0 && threadIdx.x == 0) finish_sequence(a, s, count);
  if (slice == 2 * a.pieces) {
    move_scores(a, s, g, n);
  } else {
    const int part = a.row_bytes / 16 / a.pieces;
    move_columns(a, s, g, (slice < a.pieces ? a.c.k : a.c.v) + (slice % a.pieces) * part * 16, part,
                 n);
  }
}

// Grid: (kMoveThreads rows, head, sequence). VECS: 16-byte pieces of a row.
template <int VECS>
__global__ void __launch_bounds__(kMoveThreads, VECS == 16 ? 4 : 6)
    evict_spread_kernel(const __grid_constant__ EvictArgs a) {
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const int g = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0) finish_sequence(a, s, a.counts[s]);
  const int i = blockIdx.x * kMoveThreads + threadIdx.x;
  // behind the kept positions stands -1: no count is waited for
  const int j = i < a.most ? a.keep[((int64_t)s * a.c.hkv + g) * a.budget + i] : -1;
  int64_t from = -1, at = -1;
  if (j >= 0) {
    if (a.scores_apart)
      a.scores_out[s * a.os + g * a.oh + i] = a.scores_in[s * a.ss + g * a.sh + j];
    if (a.pieces == 0) {
      from = paged_row(a.c, a.c.table + s * a.c.table_stride, j);
      at = paged_row(a.c, a.dst_table + s * a.dst_stride, i);
      if (from < 0 || at < 0) {
        report(a.status, SA_ERR_DEVICE, kWherePagedPage);
        from = -1;
      }
    }
  }
  if (!__any_sync(~0u, from >= 0)) return;
  constexpr int R = 32 / VECS, U = VECS == 16 ? 4 : 2;  // rows of an instruction; instructions in flight
  const int64_t column = g * a.c.sh + (lane % VECS) * 16;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += R * U) {
    int64_t f[U], t[U];
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * R + lane / VECS;
      f[u] = __shfl_sync(~0u, from, r);
      t[u] = __shfl_sync(~0u, at, r);
      if (f[u] >= 0) {
        k[u] = *(const uint4*)(a.c.k + f[u] + column);
        v[u] = *(const uint4*)(a.c.v + f[u] + column);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (f[u] >= 0) {
        *(uint4*)(a.c.k + t[u] + column) = k[u];
        *(uint4*)(a.c.v + t[u] + column) = v[u];
      }
  }
}

}  // namespace

size_t cache_evict_workspace_bytes(const sa_paged_cache& c) {
  return kStatusBytes + (size_t)c.n_seq * 4;
}

cudaError_t launch_cache_evict(const sa_paged_cache& c, const sa_evict_desc& d,
                               const float* scores_in, const int32_t* dst_table, int32_t* keep,
                               float* scores_out, int32_t* lens_out, void* ws, cudaStream_t s) {
  EvictArgs a{};
  a.c = make_paged_view(c);
  const bool in_place = dst_table == nullptr || dst_table == c.page_table;
  a.scores_in = scores_in;
  a.scores_out = scores_out;
  a.dst_table = in_place ? c.page_table : dst_table;
  a.dst_stride = in_place ? c.table_stride : d.dst_table_stride;
  a.keep = keep;
  a.lens_out = lens_out;
  a.status = (DeviceStatus*)ws;
  a.counts = (int32_t*)((char*)ws + kStatusBytes);
  a.ss = d.score_strides[0];
  a.sh = d.score_strides[1];
  a.os = d.out_strides[0];
  a.oh = d.out_strides[1];
  a.budget = d.budget;
  a.sinks = d.sinks;
  a.recent = d.recent;
  a.row_bytes = c.head_dim * dtype_bytes(c.dtype);
  a.scores_apart = scores_in != scores_out;
  const int64_t rows = (int64_t)c.n_seq * c.num_kv_heads;
  const int capacity = a.c.capacity;
  a.most = d.budget < capacity ? d.budget : capacity;

  // Blocks of a row: as many as hold the longest, where the SMs have room for them.
  // More measured slower even for a few rows (8 rows of 8192: 14.2 us with one block
  // each, 15.2 with two, 16.2 with four): the cluster's barriers cost what the keys
  // save. Many rows have one block each; where the table has room for longer rows
  // than 32K, it holds 16K keys, so that two run on an SM, and reads longer rows
  // again in each pass.
  int cl = 1;
  while (cl < 8 && capacity / cl > kCachedKeys) cl *= 2;
  if (rows * cl > kSms) cl = 1;
  constexpr int kRound = kSelWarps * 128;
  const int keys = ((capacity + cl - 1) / cl + kRound - 1) / kRound * kRound;
  const bool all = keys <= kCachedKeys;
  a.cluster = cl;
  a.held = all ? keys : rows > kSms ? kCachedKeys / 2 : kCachedKeys;
  const auto select = all ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kCachedKeys * 4);
  if (e != cudaSuccess) return e;
  e = launch_early(select, dim3((unsigned)(rows * cl)), kSelThreads, (size_t)a.held * 4, s, cl, a);
  if (e != cudaSuccess) return e;

  if (in_place) {
    // slices of at least 32 bytes, as many as the SMs want
    a.pieces = 1;
    while (a.pieces * 32 < a.row_bytes && rows * a.pieces * 2 < 2 * kSms) a.pieces *= 2;
  }
  if (!in_place || a.scores_apart) {
    const dim3 grid((a.most + kMoveThreads - 1) / kMoveThreads, c.num_kv_heads, c.n_seq);
    const auto spread = a.row_bytes == 256   ? evict_spread_kernel<16>
                        : a.row_bytes == 128 ? evict_spread_kernel<8>
                                             : evict_spread_kernel<4>;
    e = launch_early(spread, grid, kMoveThreads, 0, s, 1, a);
    if (e != cudaSuccess) return e;
  }
  if (in_place || !a.scores_apart) {
    const dim3 grid(2 * a.pieces + (a.scores_apart ? 0 : 1), c.num_kv_heads, c.n_seq);
    e = launch_early(evict_in_place_kernel, grid, kMoveThreads, 0, s, 1, a);
  }
  return e;
}

}  // namespace sa
