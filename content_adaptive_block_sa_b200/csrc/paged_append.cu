// Writes new keys and values into a paged cache.
//
// Row i of sequence s's new tokens goes to position len[s] - n[s] + i, as it is
// or as e4m3(x / scale). A copy with one table look-up per token: bound by memory
// for prompts (8 ragged prompts, 77K tokens of 8 x 128 values into e4m3: 84 us, 5.6
// TB/s of reads and writes), by the launch for a decode step (16 tokens: 3.1 us).
//
// One launch does it all: block 0 checks every sequence's range and pages and
// is the only writer of the status word, so that no clearing pass is needed;
// the other blocks skip, on their own, the rows that it reports. They find a row's
// sequence by bisection, which may miss one where the starts do not ascend; block
// 0 sees that and then writes the rows of every valid range itself.
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  PagedView c;
  const char* k;
  const char* v;
  int64_t kst, ksh, vst, vsh;  // byte strides: token, head
  const int32_t* cu;
  float* scores;
  int64_t scs, sch;
  int n_tokens;
  DeviceStatus* status;
};

// The new rows of sequence s: [first, last) of the input, at positions
// len - (last - first) .. ; false where the range is not a valid one.
__device__ __forceinline__ bool new_rows(const AppendArgs& a, int s, int len, int* first, int* last) {
  if (a.cu == nullptr) {
    *first = s;
    *last = s + (len > 0 ? 1 : 0);
    return true;
  }
  *first = a.cu[s];
  *last = a.cu[s + 1];
  return *first >= 0 && *first <= *last && *last <= a.n_tokens && *last - *first <= len;
}

// 16 bytes of the cache from a row's elements [e, e + 16 / size).
template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// e4m3(x / scale) of sixteen values. A quotient costs a dozen instructions, and
// 32 of them a lane would bound the kernel above the memory's time. So the values
// are multiplied by the reciprocal made a little smaller and a little larger: the
// two products enclose the quotient (reciprocal and product are off by 2^-24 each,
// the factors by 2^-21), and rounding is monotone, so where both round to the same
// e4m3 values the quotient does too. One value in about 10^5 is divided.
__device__ __forceinline__ uint4 round16(const float* q) {
  uint4 out;
  __nv_fp8x2_storage_t* y = (__nv_fp8x2_storage_t*)&out;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return out;
}

template <typename T>
__device__ __forceinline__ uint4 quantize16(const uint4* in, float scale) {
  const T* x = (const T*)in;
  const float r = 1.f / scale, less = r * (1.f - 0x1p-21f), more = r * (1.f + 0x1p-21f);
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = to_float(x[i]) * less;
  uint4 out = round16(q);
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = to_float(x[i]) * more;
  const uint4 other = round16(q);
  const bool same = ((out.x ^ other.x) | (out.y ^ other.y) | (out.z ^ other.z) | (out.w ^ other.w)) == 0;
  // reciprocals that are normal numbers only
  if (!same || !(fabsf(scale) >= 0x1p-100f && fabsf(scale) <= 0x1p100f)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = to_float(x[i]) / scale;
    out = round16(q);
  }
  return out;
}

// The check of every sequence's length, range and pages, by one block: a lane
// takes a sequence and its one or two pages, a warp the pages of a longer range.
// Tells whether the ranges' starts descend anywhere.
__device__ bool check_block(const AppendArgs& a) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  bool descends = false;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  int mine = 0;
  for (int s0 = threadIdx.x - lane; s0 < a.c.n_seq; s0 += kThreads) {
    const int s = s0 + lane;
    int p0 = 0, np = 0;
    if (s < a.c.n_seq) {
      bool bad_len = false;
      const int len = paged_len(a.c, s, &bad_len);
      if (bad_len) mine = kWherePagedLen;
      int first, last;
      const bool ok = new_rows(a, s, len, &first, &last);
      if (!ok || (s == 0 && first != 0)) mine = kWherePagedRange;
      descends |= first > last;
      if (ok && last > first) {
        p0 = (len - (last - first)) / a.c.page_size;
        np = (len - 1) / a.c.page_size - p0 + 1;
      }
      const int32_t* row = a.c.table + s * a.c.table_stride + p0;
      if (np >= 1 && (unsigned)row[0] >= (unsigned)a.c.n_pages) mine = kWherePagedPage;
      if (np >= 2 && (unsigned)row[1] >= (unsigned)a.c.n_pages) mine = kWherePagedPage;
    }
    for (unsigned rest = __ballot_sync(~0u, np > 2); rest; rest &= rest - 1) {
      const int l = __ffs(rest) - 1;
      const int32_t* row = a.c.table + (s0 + l) * a.c.table_stride + __shfl_sync(~0u, p0, l);
      const int n = __shfl_sync(~0u, np, l);
#pragma unroll 4
      for (int i = 2 + lane; i < n; i += 32)
        if ((unsigned)row[i] >= (unsigned)a.c.n_pages) mine = kWherePagedPage;
    }
  }
  if (mine) atomicMax(&bad, mine);
  descends = __syncthreads_or(descends);
  if (threadIdx.x == 0) {
    a.status->code = bad ? SA_ERR_DEVICE : SA_OK;
    a.status->where = bad;
  }
  return descends;
}

// Row t of the input to position `pos` of sequence s, by a warp: one look-up, then
// the pieces of all its heads. T: the new rows' type where the cache is e4m3; char:
// the cache's own type, copied. kVecs: 16-byte pieces of a cache row.
template <typename T, int kVecs>
__device__ __forceinline__ void put_row(const AppendArgs& a, int s, int64_t t, int pos) {
  constexpr int kIn = sizeof(T) == 1 ? 1 : 2;  // 16-byte pieces of the new row for one of the cache's
  const int lane = threadIdx.x & 31, pieces = a.c.hkv * kVecs;
  const int64_t at = paged_row(a.c, a.c.table + s * a.c.table_stride, pos);
  if (at < 0) return;
  // a copy takes two pieces of a lane at once; the quotients leave registers for one
  constexpr int U = sizeof(T) == 1 ? 2 : 1;
  for (int p0 = lane; p0 < pieces; p0 += 32 * U) {
    uint4 k[U][kIn], v[U][kIn];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + 32 * u, h = p / kVecs, vec = p % kVecs;
      if (p >= pieces) continue;
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        k[u][i] = ((const uint4*)(a.k + t * a.kst + h * a.ksh))[vec * kIn + i];
        v[u][i] = ((const uint4*)(a.v + t * a.vst + h * a.vsh))[vec * kIn + i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + 32 * u, h = p / kVecs, vec = p % kVecs;
      if (p >= pieces) continue;
      const int64_t to = at + h * a.c.sh + vec * 16;
      if constexpr (sizeof(T) == 1) {
        *(uint4*)(a.c.k + to) = k[u][0];
        *(uint4*)(a.c.v + to) = v[u][0];
      } else {
        *(uint4*)(a.c.k + to) = quantize16<T>(k[u], a.c.k_scale ? a.c.k_scale[h] : 1.f);
        *(uint4*)(a.c.v + to) = quantize16<T>(v[u], a.c.v_scale ? a.c.v_scale[h] : 1.f);
      }
    }
  }
  if (a.scores != nullptr)
    for (int h = lane; h < a.c.hkv; h += 32) a.scores[s * a.scs + h * a.sch + pos] = 0.f;
}

// Every valid range by one block, whatever the order of the ranges: a row that two
// of them name goes to both. Where another block has written a row too, it wrote
// the same. An input that is reported as bad may be slow.
template <typename T, int kVecs>
__device__ __noinline__ void put_every_range(const AppendArgs& a) {
  for (int s = 0; s < a.c.n_seq; ++s) {
    bool bad = false;
    const int len = paged_len(a.c, s, &bad);
    int first, last;
    if (!new_rows(a, s, len, &first, &last)) continue;
    for (int64_t t = first + (int)(threadIdx.x >> 5); t < last; t += kThreads / 32)
      put_row<T, kVecs>(a, s, t, len - (last - (int)t));
  }
}

template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  wait_for_earlier_kernels();
  let_next_kernel_start();
  if (blockIdx.x == 0) {
    if (check_block(a)) put_every_range<T, kVecs>(a);
    return;
  }
  constexpr int kWarps = kThreads / 32;
  const int step = (gridDim.x - 1) * kWarps;
  for (int64_t t = (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5); t < a.n_tokens; t += step) {
    int s = (int)t;
    if (a.cu != nullptr) {  // the last sequence that starts at or before row t
      int lo = 0, hi = a.c.n_seq;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid; else hi = mid;
      }
      s = lo;
    }
    if (s >= a.c.n_seq) continue;
    bool bad = false;
    const int len = paged_len(a.c, s, &bad);
    int first, last;
    if (!new_rows(a, s, len, &first, &last) || t < first || t >= last) continue;
    put_row<T, kVecs>(a, s, t, len - (last - (int)t));
  }
}

template <typename T, int kVecs>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  const int blocks = (a.n_tokens + kThreads / 32 - 1) / (kThreads / 32);
  return launch_early(paged_append_kernel<T, kVecs>, dim3(1 + (blocks < 148 * 16 ? blocks : 148 * 16)),
                      kThreads, 0, s, 1, a);
}

}  // namespace

cudaError_t launch_paged_append(const sa_paged_cache& c, const sa_paged_append_desc& d,
                                const void* k_new, const void* v_new, const int32_t* cu_new,
                                float* scores, void* ws, cudaStream_t s) {
  AppendArgs a{};
  a.c = make_paged_view(c);
  const int64_t e = dtype_bytes(d.dtype);
  a.k = (const char*)k_new;
  a.v = (const char*)v_new;
  a.kst = d.k_strides[0] * e;
  a.ksh = d.k_strides[1] * e;
  a.vst = d.v_strides[0] * e;
  a.vsh = d.v_strides[1] * e;
  a.cu = cu_new;
  a.scores = scores;
  a.scs = d.score_strides[0];
  a.sch = d.score_strides[1];
  a.n_tokens = d.n_tokens;
  a.status = (DeviceStatus*)ws;
  if (c.dtype != d.dtype) {
    if (d.dtype == SA_DTYPE_BF16)
      return c.head_dim == 128 ? launch<__nv_bfloat16, 8>(a, s) : launch<__nv_bfloat16, 4>(a, s);
    return c.head_dim == 128 ? launch<__half, 8>(a, s) : launch<__half, 4>(a, s);
  }
  switch (c.head_dim * (int)e) {
    case 64: return launch<char, 4>(a, s);
    case 128: return launch<char, 8>(a, s);
    default: return launch<char, 16>(a, s);
  }
}

}  // namespace sa
