// Attention of one new token per sequence over a paged cache.
//
// x_hj = q_h . k_j * scale over the visible positions, LSE_h = log sum_j e^x_hj,
// O_h = sum_j e^(x_hj - LSE_h) v_j; on request each position's weights, summed
// over the query heads of its group, are added to its accumulated weight.
//
// Every key and value is read once and used rep = Hq / Hkv times, so the bound
// is memory: 2 d bytes(type) per position and key/value head.
//
// The work is cut evenly however the lengths lie: the tiles (64 keys of 256-byte
// rows, 128 or 256 of shorter ones) of one (sequence, key/value head) are an item,
// all items form one list, and each block takes a contiguous part of it. A block
// whose part ends inside an item leaves a partial result (running maximum, sum,
// unnormalised O); the second kernel joins those in the order of the blocks, the
// third adds the weights. The lengths are read on the device, so that a captured
// call follows them and the host never waits.
//
// Inside a block each warp owns a quarter of a tile: 8 KB of keys and values in a
// ring of its own (cp.async, 16 bytes a lane, rows past the end or on a bad page
// filled with zeros), so that the main loop has no barrier between warps.
// Both products run on the warp's matrix instructions with keys (then output
// dimensions) on the 16-row side and the group's query heads on the 8-column
// side: S^T = K Q^T, O^T += V^T P^T. The tile form of the 5th-generation tensor
// cores wants 64 or more rows and its operands in shared memory; here a warp
// multiplies its own 16 keys without waiting for others, and at 8 columns the
// products keep the tensor pipe 15% busy while memory runs at the rate of a copy.
//
// Measured (B200; calls in a graph): 16 sequences of 65537..131072 positions, 32
// query and 8 key/value heads, bf16: 852 us, 7.2 TB/s; one of 131072: 90 us, 6.0
// TB/s; one of 1777: 8.3 us, bound by the two kernels' start and the chain length ->
// page -> row -> products -> join; 24 e4m3 sequences of up to 32768, 64 / 8 heads:
// 122 us, 6.2 TB/s; 96 fp16 sequences of 3..2048, 12 / 12 heads of 64: 59 us, 5.3
// TB/s. About 7 us of every call are its start, its join and the SMs' unequal ends.
// More than 16 query heads a key/value head read its keys and values once for every
// 16 (8 sequences of 32768, 128 / 1 heads: 155 us).
// Tried and not kept: a worker per warp (no faster, four times the partial
// results), three blocks an SM with two stages (e4m3 and long bf16 items 2 to 5%
// slower), values loaded on their own after the keys (the look-ups double).
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kStageBytes = 8192;  // a warp's keys and values of one tile
constexpr int kCtasPerSm = 2;
constexpr int kSms = 148;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// A running reference is raised when a logit passes it by 2^kLazy: until then the
// weights grow to 2^kLazy at most, which costs fp32 sums and 16-bit weights no
// precision, and most tiles skip the exchange of maxima and the rescaling.
constexpr float kLazy = 8.f;
// Weights in fp16 are taken 2^kRoom larger, by a reference that far below the
// maximum: the largest is 2^15, and those down to 2^-21 of the maximum are normal
// numbers, rounded by 2^-11. What an fp16 value leaves of a smaller one (2^-14 is
// the least normal number, the rest at most 2^-25) is multiplied by kRest, which
// makes it 2^15 at most, and goes through a product of its own: so a weight keeps
// 2^-11 down to 2^-61 of the maximum. Without it many small weights are lost
// together: behind a first key that takes all of the weight and gives nothing, the
// sum over equal keys 16 nats lower was off by 6%, and zero from 17.4 nats on.
// Measured (a captured call): 24 e4m3 sequences of up to 32768: 121.5 us without,
// 122.3 with; with logits so far apart that every tile takes the second product
// 133.5; 96 fp16 sequences of 3..2048: 58.0, 58.7, 60.6.
constexpr float kRoom = 7.f, kLeastNormal = -14.f, kRest = 0x1p40f;

struct DecodeArgs {
  PagedView c;
  const void* q;
  void* o;
  float* lse;
  const float* scores_in;
  float* scores_out;
  DeviceStatus* status;
  int32_t* errors;   // [blocks]
  float* part_o;     // [2 * blocks][columns][D]
  float* part_ml;    // [2 * blocks][columns][2]
  int2* ranges;      // [n_seq][Hkv][column tiles] first and last block of an item
  int2* ends;        // [blocks] sequence and item that a block ends but did not begin; -1
  float* logits;     // [n_seq][Hkv][most][rep] in units of log2, where weights are wanted
  int64_t qs, qh, os, oh, scs, sch;
  int hq, rep, window, sinks, most;
  bool join_by_block;
  bool carry;        // scores_out receives scores_in behind the lengths too
  bool q_by_2, o_by_4;  // rows of q on 4-byte, of o on 8-byte boundaries
  int col_tiles;     // tiles of query heads per key/value head
  int workers;       // blocks that are resident at once
  int blocks;        // of the first kernel
  int tile;          // keys of a tile
  float scale2;      // softmax scale * log2(e)
};

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(there ? 16 : 0), "l"(policy)
               : "memory");
}
// Keys and values that one worker reads once leave the L2 cache first, so that
// queries, logits and partial results stay; more tiles of columns read them again.
__device__ __forceinline__ uint64_t stream_policy(bool once) {
  uint64_t p;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two 16 x 16 tiles of bytes, transposed: a lane's r[0] and r[1] (r[2] and r[3] of
// the second tile) hold rows 4 t .. 4 t + 3 of columns g and g + 8 (g = lane / 4,
// t = lane % 4). Lane i gives the address of row i % 16 of tile i / 16.
__device__ __forceinline__ void ldsm_t8(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <typename M>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<M, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

template <typename M>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (std::is_same<M, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&h;
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&h;
  }
}
// Two e4m3 values (the low 16 bits) as a pair of fp16: exact.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffff), __NV_E4M3);
  return *(const uint32_t*)&h;
}

// Byte offset of 16-byte piece c of row r in a stage whose rows are RB bytes.
// The pieces are permuted so that the eight rows (or row pairs) that one
// shared-memory access touches lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if constexpr (RB == 64) {
    const int line = r >> 1;
    return line * 128 + (((r & 1) * 4 + c) ^ ((line & 3) << 1)) * 16;
  } else {
    return r * RB + (c ^ (r & 7)) * 16;
  }
}

// ------------------------------------------------------------- work list
// The list is cut by cost: an item of n tiles costs n + kItemCost units, for its
// query, its join and its output. The cost's units come first, then one for each
// tile. Measured with 1, 2, 3, 4: 96 sequences of 3..2048: 69, 61, 59, 59 us; 256
// of 1..600: 104, 92, 84, 84 us; equal lengths do not change.
constexpr int kItemCost = 3;

// A place in the list: tile t of item `item` (key/value head, then column tile)
// of sequence s.
struct Cursor {
  int s, item, t, tiles;
  int first, lo, count;  // the visible positions of the sequence
  int left;              // units of the worker from this tile on; none: it is not the worker's
  const int32_t* pages;  // the sequence's row of the page table

  __device__ __forceinline__ void at_sequence(const DecodeArgs& a, int seq) {
    s = seq;
    pages = a.c.table + s * a.c.table_stride;
    bool bad = false;
    const Visible v(paged_len(a.c, s, &bad), a.window, a.sinks);
    first = v.first;
    lo = v.lo;
    count = v.count;
    tiles = (count + a.tile - 1) / a.tile;
  }
  __device__ __forceinline__ void next(const DecodeArgs& a) {
    --left;
    if (++t < tiles) return;
    left -= kItemCost;
    t = 0;
    if (left <= 0 || ++item < a.c.hkv * a.col_tiles) return;
    item = 0;
#pragma unroll 1
    do {
      if (s + 1 >= a.c.n_seq) {  // never, while the lengths stand
        left = 0;
        return;
      }
      at_sequence(a, s + 1);
    } while (tiles == 0);
  }
};

// The list's units are dealt out in levels, each an equal part to every worker,
// the last level as large as the one before. Blocks start in the order of their
// number, so a worker's place that is done early takes a part of the next level:
// SMs differ in how fast memory serves them (with equal parts the fastest of them
// ended after 700 us, the slowest after 940, on 16 sequences of up to 131072).
// A part costs its block's start and its share of the join, so short lists have
// one level, and lists of few items, whose rows are joined from many parts, need
// to be longer. Measured, in units of a worker's place (items): 56 (8): 91 us with
// one level, 94 with two, 105 with four; 60 (256): 93.5, 92; 79 (192): 126, 122.5;
// 92 (64): 162, 155; 110 (16): 172, 167, 171; 220: 332, 317, 314; 664: 937, 880, 852
// and 848 with five.
constexpr int kLevels = 5;
constexpr int kTwoLevels = 40, kTwoLevelsFewItems = 96, kFourLevels = 192, kFiveLevels = 384;
constexpr int kFewItems = 8;  // workers per item that make items few

struct Levels {
  int n, shift;  // levels; the first leaves units >> shift
  __device__ __forceinline__ Levels(const DecodeArgs& a, int64_t units, int most) {
    const int64_t each = units / a.workers;
    const bool few = (int64_t)a.c.n_seq * a.c.hkv * a.col_tiles * kFewItems < a.workers;
    n = each >= kFiveLevels ? 5 : each >= kFourLevels ? 4
        : each >= (few ? kTwoLevelsFewItems : kTwoLevels) ? 2 : 1;
    n = min(n, most);
    shift = n > 2 ? 2 : each >= kTwoLevelsFewItems ? 3 : 4;
  }
  // Where a level begins: 3/4, 7/8 or 15/16 of the list for the second, half of
  // the rest further on for each one after it.
  __device__ __forceinline__ int64_t begin(int64_t units, int level) const {
    return level == 0 ? 0 : level >= n ? units : units - (units >> (level - 1 + shift));
  }
};

// A block's part of the list: its first unit and how many.
struct Part {
  int64_t start;
  int units;
  __device__ __forceinline__ Part(const DecodeArgs& a, int64_t total) {
    const Levels levels(a, total, gridDim.x / a.workers);
    const int level = blockIdx.x / a.workers, w = blockIdx.x % a.workers;
    const int64_t from = levels.begin(total, level), to = levels.begin(total, level + 1);
    // an equal share of the level, one unit more for the first ones
    const int64_t n = level < levels.n ? to - from : 0;
    const int64_t base = n >> 32 == 0 ? (uint32_t)n / a.workers : n / a.workers;
    const int64_t rest = n - base * a.workers;
    start = from + w * base + min((int64_t)w, rest);
    units = (int)(base + (w < rest ? 1 : 0));
  }
};

// Tiles and the item's cost of a sequence of n visible positions; nothing for none.
__device__ __forceinline__ int item_units(const DecodeArgs& a, int n) {
  return n ? (n + a.tile - 1) / a.tile + kItemCost : 0;
}

// Puts the cursor on unit `at` (of `units` an item) of sequence s.
__device__ __forceinline__ void put_cursor(const DecodeArgs& a, Cursor* in, int s, int64_t at, int units,
                                           int left) {
  in->at_sequence(a, s);
  in->item = at >> 32 == 0 ? (int)((uint32_t)at / (uint32_t)units) : (int)(at / units);
  const int unit = (int)(at - (int64_t)in->item * units);
  in->t = max(0, unit - kItemCost);
  in->left = left - max(0, kItemCost - unit);
}

// Puts the cursor on this block's first tile, and tells whether a length is bad.
// Up to 32 sequences every warp finds it alone; more are summed in strips, one a
// thread, by the whole block.
__device__ __forceinline__ bool find_start(const DecodeArgs& a, Cursor* in) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = a.c.hkv * a.col_tiles;
  bool bad = false;
  auto units_of = [&](int s) {
    return item_units(a, Visible(paged_len(a.c, s, &bad), a.window, a.sinks).count);
  };
  auto scan = [&](int64_t x) {
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, x, i);
      if (lane >= i) x += y;
    }
    return x;
  };
  in->left = 0;
  if (a.c.n_seq <= 32) {
    const int units = lane < a.c.n_seq ? units_of(lane) : 0;
    const int64_t mine = (int64_t)units * per_seq, upto = scan(mine);
    const Part part(a, __shfl_sync(~0u, upto, 31));
    const bool here = part.start >= upto - mine && part.start < upto;
    const int s = __ffs(__ballot_sync(~0u, here)) - 1;
    if (part.units > 0 && s >= 0)
      put_cursor(a, in, s, part.start - __shfl_sync(~0u, upto - mine, s), __shfl_sync(~0u, units, s),
                 part.units);
    return bad;
  }
  __shared__ int64_t sums[kWarps], start_at;
  __shared__ int start_s;
  const int strip = (a.c.n_seq + kThreads - 1) / kThreads;
  const int s0 = tid * strip, s1 = min(s0 + strip, a.c.n_seq);
  int64_t mine = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) mine += (int64_t)units_of(s) * per_seq;
  const int64_t upto = scan(mine);
  if (lane == 31) sums[warp] = upto;
  if (tid == 0) start_s = 0, start_at = 0;
  __syncthreads();
  int64_t total = 0, at = upto - mine;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += sums[i];
    total += sums[i];
  }
  const Part part(a, total);
  if (at <= part.start && part.start < at + mine) {
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const int64_t n = (int64_t)units_of(s) * per_seq;
      if (part.start < at + n) {
        start_s = s;
        start_at = part.start - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int units = units_of(start_s);
  if (part.units > 0 && units > 0) put_cursor(a, in, start_s, start_at, units, part.units);
  return bad;
}

// What a stage of a warp's ring holds.
struct Staged {
  uint64_t there;  // keys that are
  int s, item, t;
  int last;        // the item's last tile
};

// Q: type of q and o; T: of the cache; D: head dimension; NT: 8-column tiles of
// query heads that a worker holds.
template <typename Q, typename T, int D, int NT>
struct Geometry {
  static constexpr int RB = D * (int)sizeof(T);        // bytes of a row
  static constexpr int KPW = kStageBytes / 2 / RB;     // keys of a warp
  static constexpr int MT = KPW / 16;
  static constexpr int TILE = KPW * kWarps;
  static constexpr int COLS = 8 * NT;
  static constexpr int JOIN_ROW = D + 4;           // floats; 4: columns in different banks
  static constexpr int JOIN = kWarps * 8 * JOIN_ROW;   // floats
  static constexpr size_t SMEM =
      (size_t)kWarps * kStages * kStageBytes + JOIN * 4 + kWarps * kStages * sizeof(Staged);
};

template <typename Q, typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_decode_kernel(const __grid_constant__ DecodeArgs a) {
  using Geo = Geometry<Q, T, D, NT>;
  constexpr bool kFp8 = sizeof(T) == 1;
  using M = typename std::conditional<kFp8, __half, T>::type;  // type of the products
  constexpr int RB = Geo::RB, KPW = Geo::KPW, MT = Geo::MT, TILE = Geo::TILE;
  constexpr int KS = D / 16;              // steps along d of S, row tiles of O^T
  constexpr int KR = (KPW + 31) / 32;     // keys of a lane when it looks up rows
  constexpr int CPR = RB / 16;            // 16-byte pieces of a row
  constexpr int RPI = 32 / CPR;           // rows that a warp's copy instruction covers
  extern __shared__ __align__(128) unsigned char smem[];
  float* join_o = (float*)(smem + kWarps * kStages * kStageBytes);
  Staged* const staged = (Staged*)(join_o + Geo::JOIN) + threadIdx.x / 32 * kStages;
  __shared__ int error;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;  // row group and column pair of a fragment
  if (tid == 0) error = 0;
  __syncthreads();
  wait_for_earlier_kernels();
  let_next_kernel_start();
  Cursor in;  // of the copies
  const bool bad = find_start(a, &in);
  if (bad) error = kWherePagedLen;
  {
    const int worker = blockIdx.x;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * kStageBytes;

    // ---- copies: the page numbers of a tile are fetched one tile ahead
    const uint64_t policy = stream_policy(a.col_tiles == 1);
    int page[KR], slot[KR];
    auto look_up = [&]() {
#pragma unroll
      for (int i = 0; i < KR; ++i) {
        const int r = lane + 32 * i, c = in.t * TILE + warp * KPW + r;
        page[i] = -1;
        if (r < KPW && c < in.count) {
          const int pos = c < in.first ? c : c - in.first + in.lo;
          const int n = a.c.by_page(pos);
          slot[i] = pos - n * a.c.page_size;
          page[i] = in.pages[n];
          if ((unsigned)page[i] >= (unsigned)a.c.n_pages) page[i] = -2;
        }
      }
    };
    auto copy = [&](int stage) {
      constexpr uint32_t kNone = ~0u;
      uint32_t off[KR];
      uint64_t there = 0;
#pragma unroll
      for (int i = 0; i < KR; ++i) {
        if (page[i] == -2) error = kWherePagedPage;
        there |= (uint64_t)__ballot_sync(~0u, page[i] >= 0) << (32 * i);
        off[i] = page[i] >= 0 ? page[i] * a.c.sp_units + slot[i] * a.c.ss_units : kNone;
      }
      if (lane == 0) {
        staged[stage].there = there;
        staged[stage].s = in.s;
        staged[stage].item = in.item;
        staged[stage].t = in.t;
        staged[stage].last = in.t + 1 == in.tiles;
      }
      const uint32_t to = ring + stage * kStageBytes;
      const int head = a.col_tiles == 1 ? in.item : in.item / a.col_tiles;
      const int64_t column = head * a.c.sh + (lane % CPR) * 16;
      const char* const k = a.c.k + column;
      const char* const v = a.c.v + column;
#pragma unroll
      for (int i = 0; i < KPW / RPI; ++i) {
        const int r = i * RPI + lane / CPR;
        const uint32_t o = __shfl_sync(~0u, off[i * RPI / 32], r & 31);
        const bool is = o != kNone;
        const uint64_t from = (uint64_t)(is ? o : 0u) * a.c.unit;
        const uint32_t d = to + piece_at<RB>(r, lane % CPR);
        cp16(d, k + from, is, policy);
        cp16(d + kStageBytes / 2, v + from, is, policy);
      }
    };

    // ---- the item's query fragments and running state
    uint32_t q[NT][KS][2];
    float mul[NT][2];           // logit per product, log2 units, of columns 2 t4 and 2 t4 + 1
    float m[NT][2], l[NT][2];   // running reference (log2), this lane's part of the sum
    float o[NT][KS][4];
    int rows_h = 0;             // first query head of the item
    int cols = 0;               // query heads of the item
    int kv_head = 0, ct = 0;    // its key/value head and column tile
    int seq = 0, item = 0;
    int2 ends = make_int2(-1, -1);
    // a row of q in pairs, in the order of the products' steps; all loads of a
    // branch are under way before the first is used
    auto load_q = [&](int of, int it, int n, uint32_t (*raw)[2]) {
      const int col = n * 8 + g8, r = it % a.col_tiles * Geo::COLS + col;
      const uint16_t* row = (const uint16_t*)a.q + of * a.qs + (it / a.col_tiles * a.rep + r) * a.qh;
      auto at = [&](int k, int e) { return kFp8 ? t4 * (D / 4) + k * 4 + e * 2 : k * 16 + e * 8 + t4 * 2; };
#pragma unroll
      for (int k = 0; k < KS; ++k) raw[k][0] = raw[k][1] = 0;
      if (r >= a.rep) return;
      if (a.q_by_2) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) raw[k][e] = *(const uint32_t*)(row + at(k, e));
      } else {
        uint16_t lo[KS][2], hi[KS][2];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            lo[k][e] = row[at(k, e)];
            hi[k][e] = row[at(k, e) + 1];
          }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) raw[k][e] = lo[k][e] | (uint32_t)hi[k][e] << 16;
      }
    };
    // one tile of columns leaves the registers to fetch an item's rows when the
    // copies reach it, ahead of its keys: behind them they would queue for microseconds
    uint32_t early[KS][2];
    int early_s = -1, early_item = 0;
    auto start_item = [&]() {
      kv_head = a.col_tiles == 1 ? item : item / a.col_tiles;
      ct = item - kv_head * a.col_tiles;
      rows_h = kv_head * a.rep + ct * Geo::COLS;
      cols = min(Geo::COLS, a.rep - ct * Geo::COLS);
      const float ks = a.c.k_scale ? a.c.k_scale[kv_head] : 1.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t raw[KS][2];
        if (NT == 1 && early_s == seq && early_item == item) {
#pragma unroll
          for (int k = 0; k < KS; ++k) raw[k][0] = early[k][0], raw[k][1] = early[k][1];
        } else {
          load_q(seq, item, n, raw);
        }
        early_s = -1;
        float norm = 1.f;
        if constexpr (kFp8 && std::is_same<Q, __nv_bfloat16>::value) {
          // bf16 queries as fp16: a power of two brings the largest value of the
          // row to 2^10, so that every value above 2^-25 of it is exact
          float x[KS][4], top = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[k][e] = __uint_as_float(e & 1 ? raw[k][e >> 1] & 0xffff0000u : raw[k][e >> 1] << 16);
              top = fmaxf(top, fabsf(x[k][e]));
            }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const uint32_t ex = max((int)(__float_as_uint(top) >> 23) - 10, 1);
          norm = __uint_as_float(ex << 23);
          const float inv = __uint_as_float((254 - ex) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            q[n][k][0] = pack<M>(x[k][0] * inv, x[k][1] * inv);
            q[n][k][1] = pack<M>(x[k][2] * inv, x[k][3] * inv);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) q[n][k][0] = raw[k][0], q[n][k][1] = raw[k][1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the norm of column 2 t4 + e sits with the lanes of its row group
          mul[n][e] = a.scale2 * ks * __shfl_sync(~0u, norm, (t4 * 2 + e) * 4);
          m[n][e] = -INFINITY;
          l[n][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
      }
    };

    // ---- a piece of an item is complete: join the warps, write it
    // a join row ends in its maximum and sum
    auto row_ml = [&](int w, int c) { return (float2*)(join_o + (w * 8 + c) * Geo::JOIN_ROW + D); };
    auto finish_item = [&](bool from_start, bool to_end) {
      const bool whole = from_start && to_end;
      const int part = 2 * worker + (from_start ? 1 : 0);
      const float vs = a.c.v_scale ? a.c.v_scale[kv_head] : 1.f;
      if (tid == 0) {
        int2* const range = a.ranges + (int64_t)seq * a.c.hkv * a.col_tiles + item;
        if (from_start) range->x = worker;
        if (to_end) range->y = worker;
        if (to_end && !from_start) ends = make_int2(seq, item);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 8 >= cols) break;
        // the maxima of the last join were read before its last barrier, its O is
        // read before every thread has come to the next one
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[n][e] += __shfl_xor_sync(~0u, l[n][e], 4);
          l[n][e] += __shfl_xor_sync(~0u, l[n][e], 8);
          l[n][e] += __shfl_xor_sync(~0u, l[n][e], 16);
          if (g8 == 0) *row_ml(warp, t4 * 2 + e) = make_float2(m[n][e], l[n][e]);
        }
        __syncthreads();
        // every warp brings its O to the warps' largest maximum, and to the
        // quotient where the item is whole
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = n * 8 + t4 * 2 + e;
          float2 ml[kWarps];
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            ml[w] = *row_ml(w, t4 * 2 + e);
            top = fmaxf(top, ml[w].x);
          }
          const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += ml[w].y * exp2_fast(ml[w].x - ref);
          float f = exp2_fast(m[n][e] - ref);
          if (whole) f = sum == 0.f ? 0.f : f * vs / sum;
          if (warp == 0 && g8 == 0 && col < cols) {
            if (whole)
              a.lse[seq * (int64_t)a.hq + rows_h + col] =
                  sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
            else
              *(float2*)(a.part_ml + ((int64_t)part * Geo::COLS + col) * 2) = make_float2(top, sum);
          }
          float* to = join_o + (warp * 8 + t4 * 2 + e) * Geo::JOIN_ROW;
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int d = k * 16 + r * 8 + g8;
              to[d] = o[n][k][2 * r + e] * f;
            }
        }
        __syncthreads();
        for (int i = tid; i < 8 * D / 4; i += kThreads) {
          const int c = i / (D / 4), d = i % (D / 4) * 4, col = n * 8 + c;
          if (col >= cols) break;
          float x[4] = {};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 y = *(const float4*)(join_o + (w * 8 + c) * Geo::JOIN_ROW + d);
            x[0] += y.x;
            x[1] += y.y;
            x[2] += y.z;
            x[3] += y.w;
          }
          if (whole) {
            Q* to = (Q*)a.o + seq * a.os + (int64_t)(rows_h + col) * a.oh + d;
            if (a.o_by_4) {
              *(uint2*)to = make_uint2(pack<Q>(x[0], x[1]), pack<Q>(x[2], x[3]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) put(to + e, x[e]);
            }
          } else {
            *(float4*)(a.part_o + ((int64_t)part * Geo::COLS + col) * D + d) = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
      }
    };

    // Key of row g8 + 8 r of row tile i. The transposing load of 8-bit values gives
    // a lane four keys in a row, so the tiles of S take their keys in that order.
    auto key_of = [&](int i, int r) {
      return i * 16 + (kFp8 ? (g8 >> 1) * 4 + r * 2 + (g8 & 1) : r * 8 + g8);
    };

    // ---- the loop: a copy kStages - 1 tiles ahead, then a tile's products
    int stage = 0, behind = 0, ahead = 0;  // the products' stage, the copies'; tiles between
    bool fresh = true, from_start = false;
    if (in.left > 0) look_up();
#pragma unroll 1
    for (int step = 0;; ++step) {
      if (in.left > 0) {
        if (NT == 1 && early_s < 0 && (in.t == 0 || step == 0)) {
          early_s = in.s;
          early_item = in.item;
          load_q(early_s, early_item, 0, early);
        }
        copy(ahead);
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
        ++behind;
        in.next(a);
        if (in.left > 0) look_up();
      }
      cp_commit();
      if (step < kStages - 1) continue;
      if (behind-- == 0) break;
      __syncwarp();
      const Staged now = staged[stage];
      if (fresh) {  // while the tile is on its way
        seq = now.s;
        item = now.item;
        from_start = now.t == 0;
        fresh = false;
        start_item();
      }
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint32_t ks_at = ring + stage * kStageBytes, vs_at = ks_at + kStageBytes / 2;

      // ---- S^T = K Q^T
      float s[MT][NT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
        if constexpr (kFp8) {
          // the lane's quarter of its two keys: the same dimensions of q
          uint32_t x[2][KS];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < KS / 4; ++c)
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(x[r][c * 4]), "=r"(x[r][c * 4 + 1]), "=r"(x[r][c * 4 + 2]),
                             "=r"(x[r][c * 4 + 3])
                           : "r"(ks_at + piece_at<RB>(key_of(i, r), t4 * (KS / 4) + c))
                           : "memory");
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t f[4] = {e4m3_pair(x[0][k]), e4m3_pair(x[1][k]), e4m3_pair(x[0][k] >> 16),
                                   e4m3_pair(x[1][k] >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<M>(s[i][n], f, q[n][k][0], q[n][k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            ldsm4(f, ks_at + piece_at<RB>(i * 16 + (lane & 15), k * 2 + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<M>(s[i][n], f, q[n][k][0], q[n][k][1]);
          }
        }
      }

      // ---- softmax: logits in units of log2, -inf where there is no key
      const uint64_t there = now.there;
      constexpr uint64_t kAll = KPW == 64 ? ~0ull : (1ull << KPW) - 1;
      float top[NT][2], least[NT][2];  // of the tile's keys
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n][0] = top[n][1] = -INFINITY;
        least[n][0] = least[n][1] = INFINITY;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][n][e] *= mul[n][e & 1];
            top[n][e & 1] = fmaxf(top[n][e & 1], s[i][n][e]);
            least[n][e & 1] = fminf(least[n][e & 1], s[i][n][e]);
          }
      }
      if (there != kAll) {  // an item's last tile, or a bad page
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          top[n][0] = top[n][1] = -INFINITY;
          least[n][0] = least[n][1] = INFINITY;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool is = there >> key_of(i, e >> 1) & 1;
              if (is) least[n][e & 1] = fminf(least[n][e & 1], s[i][n][e]);
              else s[i][n][e] = -INFINITY;
              top[n][e & 1] = fmaxf(top[n][e & 1], s[i][n][e]);
            }
        }
      }
      if (a.logits != nullptr) {
        const int c0 = now.t * TILE + warp * KPW;
        float* to = a.logits + (((int64_t)seq * a.c.hkv + kv_head) * a.most + c0) * a.rep + ct * Geo::COLS;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int r = key_of(i, e >> 1), col = n * 8 + t4 * 2;
              if (col >= cols || c0 + r >= a.most) continue;
              float* x = to + (int64_t)r * a.rep + col;
              if (a.rep % 2 == 0) {
                *(float2*)x = make_float2(s[i][n][e], s[i][n][e + 1]);
              } else {
                x[0] = s[i][n][e];
                if (col + 1 < cols) x[1] = s[i][n][e + 1];
              }
            }
      }
      constexpr float kBelow = std::is_same<M, __half>::value ? kRoom : 0.f;
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) raise |= top[n][e] > m[n][e] + (kLazy + kBelow);
      if (__any_sync(~0u, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[n][e];
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            x = fmaxf(x - kBelow, m[n][e]);
            const float f = x == -INFINITY ? 1.f : exp2_fast(m[n][e] - x);
            m[n][e] = x;
            l[n][e] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[n][k][e] *= f;
              o[n][k][e + 2] *= f;
            }
          }
      }
      // the weights as the second product's columns; bf16 rounds to 2^-8, so a
      // second bf16 value holds the rest (2^-16); fp16's 2^-11 is the output's own
      // step or an eighth of it, and what it cannot hold of the smallest weights is
      // added where a tile has such
      constexpr bool kTwo = std::is_same<M, __nv_bfloat16>::value;
      uint32_t p[MT][NT][2], p2[MT][NT][2];
      bool small = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float ref[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0],
                              m[n][1] == -INFINITY ? 0.f : m[n][1]};
        if constexpr (!kTwo) {
#pragma unroll
          for (int e = 0; e < 2; ++e) small |= least[n][e] < ref[e] + kLeastNormal;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][n][e] = exp2_fast(s[i][n][e] - ref[e & 1]);
            l[n][e & 1] += s[i][n][e];
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = pack<M>(s[i][n][2 * r], s[i][n][2 * r + 1]);
            p[i][n][r] = transpose8(x);
            if constexpr (kTwo)
              p2[i][n][r] = transpose8(pack<M>(s[i][n][2 * r] - __uint_as_float(x << 16),
                                               s[i][n][2 * r + 1] - __uint_as_float(x & 0xffff0000u)));
          }
        }
      }

      // V^T of the tile's 16 keys i, kPerLoad row tiles of O^T
      constexpr int kPerLoad = kFp8 ? 2 : 1;
      auto load_v = [&](int i, int k, uint32_t (*f)[4]) {
        if constexpr (kFp8) {
          uint32_t w[4];  // keys 4 t4 .. 4 t4 + 3 of dimensions g8 and g8 + 8 of tiles 2 k, 2 k + 1
          ldsm_t8(w, vs_at + piece_at<RB>(i * 16 + (lane & 15), k * 2 + (lane >> 4)));
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            f[b][0] = e4m3_pair(w[2 * b]);
            f[b][1] = e4m3_pair(w[2 * b + 1]);
            f[b][2] = e4m3_pair(w[2 * b] >> 16);
            f[b][3] = e4m3_pair(w[2 * b + 1] >> 16);
          }
        } else {
          ldsm4_t(f[0], vs_at + piece_at<RB>(i * 16 + (lane & 7) + (lane >> 4) * 8,
                                             k * 2 + ((lane >> 3) & 1)));
        }
      };
      if constexpr (!kTwo) {
        if (__any_sync(~0u, small)) {  // what fp16 leaves of the smallest weights
          uint32_t rest[MT][NT][2];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float x = s[i][n][2 * r], y = s[i][n][2 * r + 1];
                const float2 h = __half22float2(__floats2half2_rn(x, y));
                rest[i][n][r] = transpose8(pack<M>(x < 0x1p-14f ? (x - h.x) * kRest : 0.f,
                                                   y < 0x1p-14f ? (y - h.y) * kRest : 0.f));
              }
#pragma unroll
          for (int k = 0; k < KS / kPerLoad; ++k) {
            float sum[kPerLoad][NT][4] = {};
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              uint32_t f[kPerLoad][4];
              load_v(i, k, f);
#pragma unroll
              for (int b = 0; b < kPerLoad; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<M>(sum[b][n], f[b], rest[i][n][0], rest[i][n][1]);
            }
#pragma unroll
            for (int b = 0; b < kPerLoad; ++b)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][k * kPerLoad + b][e] += sum[b][n][e] * (1.f / kRest);
          }
        }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int k = 0; k < KS / kPerLoad; ++k) {
          uint32_t f[kPerLoad][4];
          load_v(i, k, f);
#pragma unroll
          for (int b = 0; b < kPerLoad; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<M>(o[n][k * kPerLoad + b], f[b], p[i][n][0], p[i][n][1]);
              if constexpr (kTwo) mma<M>(o[n][k * kPerLoad + b], f[b], p2[i][n][0], p2[i][n][1]);
            }
        }
      }

      // ---- the stage is free
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (now.last || behind == 0) {
        finish_item(from_start, now.last != 0);
        fresh = true;
      }
    }
    cp_wait<0>();
    if (tid == 0) a.ends[worker] = ends;
  }
  __syncthreads();
  if (tid == 0) a.errors[blockIdx.x] = error;
}

// ---------------------------------------------------------- second kernel
// A block per row of the output that more than one block of the first kernel
// holds a part of, or that sees nothing: its warps take the parts in turn, four
// dimensions a lane, the loads of several parts under way at once, each warp with a
// running maximum and sum of its own. One block more gathers the first kernel's errors
// into the status word.
//
// Which rows those are is found from the rows where they are few: grid (query
// head, sequence), and sequence n_seq for the status. Most rows of a large batch
// are whole, though, and looking at each costs more than joining; so there it is
// found from the blocks: an item that several share has one block that ends it
// without having begun it. Grid: (column, block), then one for the status, then
// one for eight sequences each that looks for empty ones.
constexpr int kJoinThreads = 256;

template <typename Q>
__device__ void empty_rows(const DecodeArgs& a, int s, int D) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < a.hq * D; i += 32) put((Q*)a.o + s * a.os + i / D * a.oh + i % D, 0.f);
  for (int h = lane; h < a.hq; h += 32) a.lse[(int64_t)s * a.hq + h] = -INFINITY;
}

// U: a warp's parts under way at once. Eight where the rows leave SMs idle (one
// sequence: 8.8 us a call with four, 8.3 with eight), else four, for more blocks an
// SM (96 short sequences: 58.7 us with eight, 57.8 with four).
template <typename Q, int D, int U>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int L = D / 4, W = kJoinThreads / L;  // lanes of a part; parts side by side
  __shared__ float4 part_x[W][L];
  __shared__ float2 part_ml[W];
  const int tid = threadIdx.x, l4 = tid % L, p = tid / L;
  let_next_kernel_start();
  wait_for_earlier_kernels();
  if (blockIdx.y == (a.join_by_block ? a.blocks : a.c.n_seq)) {
    int bad = 0;
    for (int i = tid; i < a.blocks; i += kJoinThreads) bad = max(bad, a.errors[i]);
    const bool page = __syncthreads_or(bad == kWherePagedPage), len = __syncthreads_or(bad != 0);
    if (blockIdx.x == 0 && tid == 0) {
      a.status->code = len ? SA_ERR_DEVICE : SA_OK;
      a.status->where = page ? kWherePagedPage : len ? kWherePagedLen : 0;
    }
    return;
  }
  const int columns = a.rep > 8 ? 16 : 8;
  int s, g, ct, r;
  int2 range;
  if (a.join_by_block) {
    const int b = blockIdx.y;
    if (b > a.blocks) {
      s = (b - a.blocks - 1) * (kJoinThreads / 32) + tid / 32;
      if (blockIdx.x == 0 && s < a.c.n_seq && a.c.lens[s] <= 0) empty_rows<Q>(a, s, D);
      return;
    }
    const int2 end = a.ends[b];
    s = end.x;
    if (s < 0) return;
    g = end.y / a.col_tiles;
    ct = end.y - g * a.col_tiles;
    r = ct * columns + blockIdx.x;
    if (r >= a.rep) return;
    range = make_int2(a.ranges[((int64_t)s * a.c.hkv + g) * a.col_tiles + ct].x, b);
  } else {
    s = blockIdx.y;
    g = blockIdx.x / a.rep;
    r = blockIdx.x - g * a.rep;
    ct = r / columns;
    range = a.ranges[((int64_t)s * a.c.hkv + g) * a.col_tiles + ct];
    // an empty sequence has no tiles: nobody wrote its range, and it has no parts
    if (a.c.lens[s] <= 0) range = make_int2(0, -1);
    if (range.x == range.y) return;  // written by its block
  }
  const int h = g * a.rep + r;
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  const int col = r - ct * columns, end = range.y;
#pragma unroll 1
  for (int w0 = range.x + p; w0 <= end; w0 += U * W) {
    float2 ml[U];
    float4 y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = w0 + u * W;
      ml[u] = make_float2(-INFINITY, 0.f);
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (w <= end) {  // the item begins in the first worker's range
        const int64_t at = (int64_t)(2 * w + (w == range.x ? 1 : 0)) * columns + col;
        ml[u] = *(const float2*)(a.part_ml + at * 2);
        y[u] = *(const float4*)(a.part_o + at * D + l4 * 4);
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float ref = top == -INFINITY ? 0.f : top, f = exp2_fast(m - ref);
    m = top;
    l *= f;
    x = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float k = exp2_fast(ml[u].x - ref);
      l += ml[u].y * k;
      x = make_float4(x.x + y[u].x * k, x.y + y[u].y * k, x.z + y[u].z * k, x.w + y[u].w * k);
    }
  }
  part_x[p][l4] = x;
  if (l4 == 0) part_ml[p] = make_float2(m, l);
  __syncthreads();
  if (tid >= D) return;
  float top = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) top = fmaxf(top, part_ml[w].x);
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
  for (int w = 0; w < W; ++w) {
    const float f = exp2_fast(part_ml[w].x - ref);
    sum += part_ml[w].y * f;
    y += ((const float*)part_x[w])[tid] * f;
  }
  const float vs = a.c.v_scale ? a.c.v_scale[g] : 1.f;
  put((Q*)a.o + s * a.os + h * a.oh + tid, sum == 0.f ? 0.f : y / sum * vs);
  if (tid == 0) a.lse[(int64_t)s * a.hq + h] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

// ----------------------------------------------------------- third kernel
// e^(x - LSE) with both in units of log2; nothing where the row sees nothing.
__device__ __forceinline__ float weight(float x, float lse2) {
  return lse2 == -INFINITY ? 0.f : exp2_fast(x - lse2);
}

constexpr int kWeightKeys = 4 * kThreads;  // positions of a block

// Adds the weights, and carries over what stands behind a length where the scores
// go to another array. Grid: (stretches of positions in turn, key/value head,
// sequence). The lengths and the scores so far are known before the earlier kernels
// have ended. The waiting comes before any block's end, so that the grid does not
// end before the kernels that it follows.
__global__ void __launch_bounds__(kThreads) paged_weights_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int U = kWeightKeys / kThreads;
  const int tid = threadIdx.x, g = blockIdx.y, s = blockIdx.z;
  bool bad = false;
  const int len = paged_len(a.c, s, &bad);
  const Visible vis(len, a.window, a.sinks);
  const float* old = a.scores_in + s * a.scs + g * a.sch;
  float* to = a.scores_out + s * a.scs + g * a.sch;
  const float* lse = a.lse + (int64_t)s * a.hq + g * a.rep;
  int j0 = blockIdx.x * kWeightKeys;
  const int end = a.carry ? a.c.capacity : len;
  if (j0 >= end) {
    wait_for_earlier_kernels();
    return;
  }
#pragma unroll 1
  for (; j0 < end; j0 += gridDim.x * kWeightKeys) {
    float w[U], was[U];
    const float* x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kThreads + tid;
      const bool seen = j < vis.first || j >= vis.lo;
      const int c = j < vis.first ? j : j - vis.lo + vis.first;
      x[u] = j < len && seen ? a.logits + (((int64_t)s * a.c.hkv + g) * a.most + c) * a.rep : nullptr;
      w[u] = 0.f;
      was[u] = j < end ? old[j] : 0.f;
    }
    wait_for_earlier_kernels();
    int i = 0;
    if (a.rep % 4 == 0) {
#pragma unroll 1
      for (; i < a.rep; i += 4) {
        float4 y[U];
        float z[4];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (x[u]) y[u] = *(const float4*)(x[u] + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = lse[i + e] * kLog2e;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (x[u])
            w[u] += (weight(y[u].x, z[0]) + weight(y[u].y, z[1])) +
                    (weight(y[u].z, z[2]) + weight(y[u].w, z[3]));
      }
    }
#pragma unroll 1
    for (; i < a.rep; ++i) {
      const float z = lse[i] * kLog2e;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (x[u]) w[u] += weight(x[u][i], z);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kThreads + tid;
      if (j < end && (x[u] || old != to)) to[j] = was[u] + w[u];
    }
  }
}

// ------------------------------------------------------------------- host
int most_visible(const sa_paged_cache& c, const sa_paged_decode_desc& d) {
  const int64_t cap = paged_capacity(c), see = (int64_t)d.window + d.sinks;
  return (int)(d.window > 0 && see < cap ? see : cap);
}

// How a call is cut, and where its workspace's parts begin.
struct Plan {
  int cols, col_tiles, workers, blocks;
  size_t errors, ends, ranges, part_o, part_ml, logits, bytes;
  Plan(const sa_paged_cache& c, const sa_paged_decode_desc& d) {
    const int rep = d.num_q_heads / c.num_kv_heads;
    cols = rep > 8 ? 16 : 8;
    col_tiles = (rep + cols - 1) / cols;
    workers = kSms * kCtasPerSm;
    // one level where even full sequences would not make more
    const int tile = kWarps * kStageBytes / 2 / (c.head_dim * dtype_bytes(c.dtype));
    const int64_t units = ((int64_t)most_visible(c, d) / tile + 1 + kItemCost) * c.n_seq *
                          c.num_kv_heads * col_tiles;
    blocks = units < (int64_t)workers * kTwoLevels ? workers : workers * kLevels;
    auto place = [this](size_t n) {
      const size_t at = bytes;
      bytes += (n + 255) / 256 * 256;
      return at;
    };
    bytes = kStatusBytes;
    errors = place((size_t)blocks * 4);
    ends = place((size_t)blocks * 8);
    ranges = place((size_t)c.n_seq * c.num_kv_heads * col_tiles * 8);
    part_ml = place((size_t)2 * blocks * cols * 8);
    part_o = place((size_t)2 * blocks * cols * c.head_dim * 4);
    logits = bytes;
    if (d.accumulate) logits = place((size_t)c.n_seq * d.num_q_heads * most_visible(c, d) * 4);
  }
};

template <typename Q, typename T, int D, int NT>
cudaError_t launch(const Plan& plan, DecodeArgs a, cudaStream_t s) {
  using Geo = Geometry<Q, T, D, NT>;
  a.tile = Geo::TILE;
  cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<Q, T, D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_early(paged_decode_kernel<Q, T, D, NT>, dim3(plan.blocks), kThreads, Geo::SMEM, s, 1, a);
  if (e != cudaSuccess) return e;
  const int columns = a.rep < plan.cols ? a.rep : plan.cols;
  a.join_by_block = (int64_t)a.c.n_seq * a.hq > (int64_t)plan.blocks * columns;
  const dim3 join = a.join_by_block ? dim3(columns, plan.blocks + 1 + (a.c.n_seq + 7) / 8)
                                    : dim3(a.hq, a.c.n_seq + 1);
  e = launch_early(a.c.n_seq * a.hq <= 2 * kSms ? paged_join_kernel<Q, D, 8> : paged_join_kernel<Q, D, 4>,
                   join, kJoinThreads, 0, s, 1, a);
  if (e != cudaSuccess || a.logits == nullptr) return e;
  // stretches of a full sequence, but no more blocks than two rounds of the SMs'
  // places (sixteen): a table made for far longer sequences would start thousands
  // that find nothing (64 sequences of 500 with room for 131072: 105 us)
  const int64_t stretches = (a.c.capacity + kWeightKeys - 1) / kWeightKeys,
                rows = (int64_t)a.c.n_seq * a.c.hkv, room = kSms * 32 / rows + 1;
  const dim3 grid((unsigned)(stretches < room ? stretches : room), a.c.hkv, a.c.n_seq);
  return launch_early(paged_weights_kernel, grid, kThreads, 0, s, 1, a);
}

template <typename Q, typename T>
cudaError_t dispatch(int d, const Plan& plan, const DecodeArgs& a, cudaStream_t s) {
  if (d == 128)
    return plan.cols == 8 ? launch<Q, T, 128, 1>(plan, a, s)
                          : launch<Q, T, 128, 2>(plan, a, s);
  return plan.cols == 8 ? launch<Q, T, 64, 1>(plan, a, s)
                        : launch<Q, T, 64, 2>(plan, a, s);
}

}  // namespace

size_t paged_decode_workspace_bytes(const sa_paged_cache& c, const sa_paged_decode_desc& d) {
  return Plan(c, d).bytes;
}

cudaError_t launch_paged_decode(const sa_paged_cache& c, const sa_paged_decode_desc& d,
                                const void* q, void* o, float* lse, const float* scores_in,
                                float* scores_out, void* ws, cudaStream_t s) {
  const Plan plan(c, d);
  DecodeArgs a{};
  a.c = make_paged_view(c);
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.scores_in = scores_in;
  a.scores_out = scores_out;
  a.carry = scores_in != scores_out && !d.keep_tail;
  char* base = (char*)ws;
  a.status = (DeviceStatus*)base;
  a.errors = (int32_t*)(base + plan.errors);
  a.ranges = (int2*)(base + plan.ranges);
  a.ends = (int2*)(base + plan.ends);
  a.part_o = (float*)(base + plan.part_o);
  a.part_ml = (float*)(base + plan.part_ml);
  a.logits = d.accumulate ? (float*)(base + plan.logits) : nullptr;
  a.qs = d.q_strides[0];
  a.qh = d.q_strides[1];
  a.os = d.o_strides[0];
  a.oh = d.o_strides[1];
  a.scs = d.score_strides[0];
  a.sch = d.score_strides[1];
  a.hq = d.num_q_heads;
  a.rep = d.num_q_heads / c.num_kv_heads;
  a.window = d.window;
  a.sinks = d.sinks;
  a.most = most_visible(c, d);
  a.q_by_2 = ((uintptr_t)q | (uintptr_t)(a.qs * 2) | (uintptr_t)(a.qh * 2)) % 4 == 0;
  a.o_by_4 = ((uintptr_t)o | (uintptr_t)(a.os * 2) | (uintptr_t)(a.oh * 2)) % 8 == 0;
  a.col_tiles = plan.col_tiles;
  a.workers = plan.workers;
  a.blocks = plan.blocks;
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.f / sqrtf((float)c.head_dim);
  a.scale2 = scale * kLog2e;
  if (c.dtype == SA_DTYPE_E4M3)
    return d.dtype == SA_DTYPE_BF16
               ? dispatch<__nv_bfloat16, __nv_fp8_e4m3>(c.head_dim, plan, a, s)
               : dispatch<__half, __nv_fp8_e4m3>(c.head_dim, plan, a, s);
  return d.dtype == SA_DTYPE_BF16 ? dispatch<__nv_bfloat16, __nv_bfloat16>(c.head_dim, plan, a, s)
                                  : dispatch<__half, __half>(c.head_dim, plan, a, s);
}

}  // namespace sa
