// Embedding lookup with a factor, and the table's gradient by sorted tokens;
// and their C calls.
//
//   out[t] = scale * table[id[t]]         (zeros where id[t] is no row)
//   dtable[v] = scale * sum of dout[t] over the tokens t with id[t] = v
//
// The gradient takes three launches.  The first sorts: every CTA owns the rows of
// one remainder (frequent tokens often have neighbouring ids), reads all ids (they
// stay in L2), counts those of lower remainders (so that it knows where its tokens
// go without asking another CTA) and places its own in the order of (row, token).
// The second sums: a run of sorted tokens at a time, with the rest of its
// last row, and writes zeros to the rows without tokens; a row of more than twice
// as many tokens is summed in parts, one a run.  The third joins the parts in order.
// Each sum has one order: the same call gives the same bits.
//
// Device times: 32768 tokens of a text (ids by 1 / id), 40960 x 2048 bf16: the lookup 32 us, 5.3
// TB/s of the rows in use and the 134 MB written; the gradient 68 us: sorting 10
// (instructions: every CTA looks at every id), sums 48 (126 MB read, 168 written:
// 6.1 TB/s), joining 7 (latency of its four dependent reads).  All tokens the same:
// 30 + 47 + 18.  5003 tokens, 1009 x 321 fp32: 16 us, latencies one after another.

#include <cmath>

#include "zero_flatstep.h"
#include "zero_embedding_internal.h"
#include "zero_rows.cuh"
#include "zero_rows_host.h"

namespace zfs {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kLookupCtas = 4;    // of an SM: four rows of 16 bytes a thread in flight
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 128;    // a power of two
constexpr int kSortRows = 1024;   // of a CTA at most: a counter for each and every warp, 128 KB
constexpr int kSortLoads = 8;     // ids in flight per lane
constexpr int kSortList = 128;    // tokens that a warp keeps, else it reads its ids again
constexpr int kLeastChunk = 8, kMostChunk = 32;  // sorted tokens of a run
constexpr int kJoinWarps = 16;

struct EmbArgs {
  long long tokens;
  int vocab, dim, lanes;       // lanes: threads on a row
  const void* ids;
  int wide_ids;
  const void* rows;            // the table, or dout
  void* out;                   // the looked up rows, or dtable
  long long row_stride, out_stride;
  float scale;
  int accumulate;
  // gradient
  int4* sorted;                // token, row, where the row's tokens begin and end, in the order of the rows
  int* counts;                 // [vocab] tokens of a row
  int* live;                   // tokens that have a row; then how many rows are in parts
  int4* heavy;                 // the rows in parts: first run, row, how many runs
  float* parts;                // [run][of a row that began before it, of its last row][pitch]
  int pitch, slabs;            // pitch: columns of a part, slabs: of 128 columns
  int remainders, per_cta;     // sorting CTAs, rows of each
  int runs, chunk;             // runs of `chunk` sorted tokens
  int columns;                 // warps for the columns of a run
};

// The row of an id, -1 if it has none.
template <typename Id>
__device__ __forceinline__ int row_of(Id id, int vocab) {
  if constexpr (sizeof(Id) == 8) {
    const unsigned low = static_cast<unsigned>(id), high = static_cast<unsigned>(static_cast<unsigned long long>(id) >> 32);
    return high == 0u && low < static_cast<unsigned>(vocab) ? static_cast<int>(low) : -1;
  } else {
    return static_cast<unsigned>(id) < static_cast<unsigned>(vocab) ? id : -1;
  }
}

template <bool kFp32, int kVec, typename Id>
__global__ void __launch_bounds__(kEmbThreads, kLookupCtas) embedding_kernel(const __grid_constant__ EmbArgs a) {
  constexpr int kRows = 4;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  const Id* ids = static_cast<const Id*>(a.ids);
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kEmbThreads / lanes;
  const long long step = static_cast<long long>(gridDim.x) * per_cta;
  const int at = blockIdx.y * lanes * 8, cols = a.dim - at;
  const long long first = static_cast<long long>(blockIdx.x) * per_cta + threadIdx.x / lanes;
  // the next ids are read while the rows of these are on their way
  Id next[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) next[i] = first + step * i < a.tokens ? ids[first + step * i] : -1;
  for (long long t0 = first; t0 < a.tokens; t0 += step * kRows) {
    int row[kRows];
    Eight<kFp32, kVec> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      row[i] = row_of(next[i], a.vocab);
      const long long after = t0 + step * (kRows + i);
      next[i] = after < a.tokens ? ids[after] : -1;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      load_eight<kFp32, kVec>(static_cast<const char*>(a.rows) + (row[i] * a.row_stride + at) * kSize, lane, lanes,
                              row[i] >= 0 ? cols : 0, &raw[i]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long t = t0 + step * i;
      if (t >= a.tokens) break;
      float x[8];
      widen_eight<kFp32, kVec>(raw[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = row[i] >= 0 ? x[k] * a.scale : 0.0f;
      store_eight<kFp32, kVec>(static_cast<char*>(a.out) + (t * a.out_stride + at) * kSize, lane, lanes, cols, x);
    }
  }
}

__device__ __forceinline__ int warp_total(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Calls f(token, row, the lanes that call it now, those of them with the same
// row) for every token of a warp's list, in order.
template <typename F>
__device__ __forceinline__ void walk_list(const int2* list, int count, F f) {
  const int lane = threadIdx.x % 32;
  for (int i = 0; i < count; i += 32) {
    const bool in = i + lane < count;
    const unsigned some = __ballot_sync(0xffffffffu, in);
    if (in) {
      const int2 e = list[i + lane];
      f(e.x, e.y, some, __match_any_sync(some, e.y));
    }
    __syncwarp();
  }
}
// The same from the ids, for a warp whose tokens do not fit its list.  rows_of: a
// CTA's rows have the remainder blockIdx.x, `row` is their quotient.
struct Share {
  long long begin, end;  // the warp's tokens
  int mask, shift;       // remainder, quotient
};
template <typename Id, typename F>
__device__ __forceinline__ void walk_ids(const EmbArgs& a, const Share& own, F f) {
  const int lane = threadIdx.x % 32;
  for (long long t = own.begin; t < own.end; t += 32) {
    const int v = t + lane < own.end ? row_of(static_cast<const Id*>(a.ids)[t + lane], a.vocab) : -1;
    const bool in = v >= 0 && (v & own.mask) == static_cast<int>(blockIdx.x);
    const unsigned some = __ballot_sync(0xffffffffu, in);
    if (in) f(static_cast<int>(t) + lane, v >> own.shift, some, __match_any_sync(some, v));
    __syncwarp();
  }
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ EmbArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int shared[];
  const Id* ids = static_cast<const Id*>(a.ids);
  __shared__ int2 lists[kSortWarps][kSortList];
  __shared__ int sums[kSortWarps];
  __shared__ int base;
  int* const counters = shared;                               // [warp][row]
  int* const begins = counters + kSortWarps * a.per_cta;      // [row], then the end of the last
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned lower = (1u << lane) - 1u;  // the lanes before this one
  const int b = blockIdx.x, shift = __ffs(a.remainders) - 1;
  const long long per_warp = (a.tokens + kSortThreads - 1) / kSortThreads * 32;
  const long long end = (warp + 1) * per_warp < a.tokens ? (warp + 1) * per_warp : a.tokens;
  const Share own{warp * per_warp, end, a.remainders - 1, shift};
  int* mine = counters + warp * a.per_cta;
  for (int i = threadIdx.x; i < kSortWarps * a.per_cta; i += kSortThreads) counters[i] = 0;
  if (b == 0 && threadIdx.x == 0) a.live[1] = 0;
  // the warp's tokens of this CTA's rows to its list; those of CTAs before it counted
  int before = 0, listed = 0;
  auto take = [&](Id id, int token) {
    const unsigned row = row_of(id, a.vocab), rest = row & own.mask;  // (unsigned)-1: none
    const bool real = row != 0xFFFFFFFFu;
    before += real && rest < static_cast<unsigned>(b);
    const bool in = real && rest == static_cast<unsigned>(b);
    const unsigned some = __ballot_sync(0xffffffffu, in);
    if (some == 0u) return;
    const int at = listed + __popc(some & lower);
    if (in && at < kSortList) lists[warp][at] = make_int2(token, static_cast<int>(row >> shift));
    listed += __popc(some);
  };
  long long t0 = own.begin;
  for (; t0 + 32 * kSortLoads <= end; t0 += 32 * kSortLoads) {
    Id id[kSortLoads];
    const Id* from = ids + t0 + lane;
#pragma unroll
    for (int u = 0; u < kSortLoads; ++u) id[u] = from[32 * u];
#pragma unroll
    for (int u = 0; u < kSortLoads; ++u) take(id[u], static_cast<int>(t0) + 32 * u + lane);
  }
  for (; t0 < end; t0 += 32) take(t0 + lane < end ? ids[t0 + lane] : -1, static_cast<int>(t0) + lane);
  before = warp_total(before);
  if (lane == 0) sums[warp] = before;
  __syncthreads();
  const bool fits = listed <= kSortList;
  auto count = [&](int, int r, unsigned, unsigned same) {
    if ((same & lower) == 0u) mine[r] += __popc(same);
  };
  if (fits) walk_list(lists[warp], listed, count);
  else walk_ids<Id>(a, own, count);
  if (warp == 0) {
    before = warp_total(sums[lane]);
    if (lane == 0) base = before;
  }
  __syncthreads();
  // where every (row, warp) begins: over the rows kSortThreads at a time
  int running = base;
  for (int r0 = 0; r0 < a.per_cta; r0 += kSortThreads) {
    const int r = r0 + threadIdx.x;
    int total = 0;
    if (r < a.per_cta) {
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = counters[w * a.per_cta + r];
        counters[w * a.per_cta + r] = total;
        total += c;
      }
    }
    int scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int before_mine = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before_mine += sums[w];
      all += sums[w];
    }
    if (r < a.per_cta) {
      begins[r] = running + before_mine + scan - total;
      const long long v = (static_cast<long long>(r) << shift) + b;
      if (v < a.vocab) a.counts[v] = total;
    }
    running += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    begins[a.per_cta] = running;
    if (b + 1 == a.remainders) a.live[0] = running;
  }
  __syncthreads();
  auto place = [&](int t, int r, unsigned some, unsigned same) {
    const int at = mine[r];
    __syncwarp(some);
    if ((same & lower) == 0u) mine[r] = at + __popc(same);
    const int begin = begins[r], to = begin + at + __popc(same & lower);
    if (ZFS_CHECK(to >= 0 && to < a.tokens)) a.sorted[to] = make_int4(t, (r << shift) + b, begin, begins[r + 1]);
  };
  if (fits) walk_list(lists[warp], listed, place);
  else walk_ids<Id>(a, own, place);
}

// What a lane of a summing warp holds: 32 bytes of vectors, eight single elements,
// or two (so that narrow tables have warps enough: below kNarrow fp32 or 2 kNarrow
// bf16 columns).
enum : int { kVectors = 8, kSingles = 1, kFewSingles = 0 };
constexpr int kNarrow = 512;
template <bool kFp32, int kMode>
constexpr int kSumParts = kMode == kVectors && !kFp32 ? 2 : 1;
template <int kMode>
constexpr int kSumCount = kMode == kFewSingles ? 2 : 8;
template <bool kFp32, int kMode>
constexpr int kSumColumns = 32 * kSumParts<kFp32, kMode> * kSumCount<kMode>;

// The warp's columns, from `at` on, of a row of the table's gradient.
template <bool kFp32, int kMode>
__device__ __forceinline__ void put_row(const EmbArgs& a, int row, int at, int lane, const float* sum) {
  constexpr long long kSize = kFp32 ? 4 : 2;
  constexpr int kVec = kMode == kVectors ? 8 : 1, kCount = kSumCount<kMode>;
  if (!ZFS_CHECK(row >= 0 && row < a.vocab)) return;
  char* to = static_cast<char*>(a.out) + (row * a.out_stride + at) * kSize;
  float x[kCount];
#pragma unroll
  for (int k = 0; k < kCount; ++k) x[k] = sum[k] * a.scale;
  if (a.accumulate) {
    Eight<kFp32, kVec, kCount> old;
    float y[kCount];
    load_eight<kFp32, kVec, kCount>(to, lane, 32, a.dim - at, &old);
    widen_eight<kFp32, kVec, kCount>(old, y);
#pragma unroll
    for (int k = 0; k < kCount; ++k) x[k] += y[k];
  }
  store_eight<kFp32, kVec, kCount>(to, lane, 32, a.dim - at, x);
}

// Rows of whole vectors come to a warp by asynchronous copies, kSumDepth (1 KB
// each) on their way: a row's address takes two dependent reads, so a warp lives
// for some latencies whatever it does, and registers would hold four.
constexpr int kSumDepth = 8;
constexpr int kSumThreads = 128, kSumWarps = kSumThreads / 32;  // few: a CTA lasts as long as its longest run
constexpr int kSumShared = kSumWarps * kSumDepth * 1024;

__host__ __device__ inline int ctas_of(long long jobs, int columns) {
  return static_cast<int>((jobs * columns + kSumWarps - 1) / kSumWarps);
}

// A warp takes kSumColumns columns of a run, or of 32 rows that may have no token.
template <bool kFp32, bool kOutFp32, int kMode>
__global__ void __launch_bounds__(kSumThreads, 6) embedding_sum_kernel(const __grid_constant__ EmbArgs a) {
  constexpr int kVec = kMode == kVectors ? 8 : 1, kParts = kSumParts<kFp32, kMode>, kCount = kSumCount<kMode>, kPart = 32 * kCount;
  constexpr long long kSize = kFp32 ? 4 : 2, kOutSize = kOutFp32 ? 4 : 2;
  const int lane = threadIdx.x % 32;
  // CTAs of runs, which wait for what they read, and of zeros, which only write, in turn
  const int zeros = a.accumulate ? 0 : (a.vocab + 31) / 32, run_ctas = ctas_of(a.runs, a.columns), zero_ctas = ctas_of(zeros, a.columns);
  const int in_turn = 2 * (run_ctas < zero_ctas ? run_ctas : zero_ctas), b = blockIdx.x;
  const bool sums = b < in_turn ? b % 2 == 0 : run_ctas > zero_ctas;
  const long long unit = static_cast<long long>(b < in_turn ? b / 2 : b - in_turn / 2) * kSumWarps + threadIdx.x / 32;
  const long long job = unit / a.columns;
  if (job >= (sums ? a.runs : zeros)) return;
  const int at = static_cast<int>(unit - job * a.columns) * kSumColumns<kFp32, kMode>, cols = a.dim - at;
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
  if (!sums) {
    const float zero[kCount] = {};
    const long long v0 = job * 32;
    unsigned empty = __ballot_sync(0xffffffffu, v0 + lane < a.vocab && a.counts[v0 + lane] == 0);
    while (empty) {
      const long long v = v0 + __ffs(empty) - 1;
      empty &= empty - 1;
#pragma unroll
      for (int n = 0; n < kParts; ++n)
        store_eight<kOutFp32, kVec, kCount>(static_cast<char*>(a.out) + (v * a.out_stride + at + n * kPart) * kOutSize, lane,
                                            32, cols - n * kPart, zero);
    }
    return;
  }
  const int run = static_cast<int>(job), heavy = 2 * a.chunk;
  const int begin = run * a.chunk;
  // a lane holds three of the entries that a run can have (32, and 63 of its last row)
  auto entry = [&](int q) {
    return static_cast<long long>(begin) + q < a.tokens ? a.sorted[begin + q] : make_int4(0, -1, 0, 0);
  };
  int4 now = entry(lane), next = entry(32 + lane);
  const int4 third = entry(64 + lane);
  const int live = a.live[0];
  if (begin >= live) return;
  const int full = begin + a.chunk < live ? a.chunk : live - begin;
  int q = 0, end = full;  // relative to begin
  // a row that began before this run: an earlier run sums it, or all in parts
  const int first_begin = __shfl_sync(0xffffffffu, now.z, 0), first_end = __shfl_sync(0xffffffffu, now.w, 0);
  if (first_begin < begin && first_end - first_begin <= heavy) q = first_end - begin;
  if (q >= end) return;
  const int last_begin = __shfl_sync(0xffffffffu, now.z, full - 1), last_end = __shfl_sync(0xffffffffu, now.w, full - 1);
  if (last_end - last_begin <= heavy) end = last_end - begin;  // the last row whole
  F2 sum[kParts][kCount / 2] = {};
  int row = -1, row_begin = 0, row_end = 0;
  auto put = [&]() {
    const bool part = row_end - row_begin > heavy;
    const int which = row_begin < begin ? 0 : 1;
    if (part && which == 1 && lane == 0 && at == 0)
      a.heavy[atomicAdd(a.live + 1, 1)] = make_int4(run, row, (row_end - 1) / a.chunk - run + 1, 0);
#pragma unroll
    for (int n = 0; n < kParts; ++n) {
      float x[kCount];
#pragma unroll
      for (int k = 0; k < kCount / 2; ++k) {
        split(sum[n][k], &x[2 * k], &x[2 * k + 1]);
        sum[n][k] = 0;
      }
      if (part) store_eight<true, kVec, kCount>(a.parts + (run * 2LL + which) * a.pitch + at + n * kPart, lane, 32,
                                                cols - n * kPart, x);
      else put_row<kOutFp32, kMode>(a, row, at + n * kPart, lane, x);
    }
  };
  const char* const rows = static_cast<const char*>(a.rows) + at * kSize;
  // a group of 32 entries at a time: where a row begins among them
  int group = 0;
  unsigned begins = 0;
  auto look = [&]() { begins = __ballot_sync(0xffffffffu, begin + group + lane == now.z); };
  auto row_at = [&](int i) {  // of this group or the next
    const int token = __shfl_sync(0xffffffffu, i - group < 32 ? now.x : next.x, i % 32);
    return rows + (ZFS_CHECK(token >= 0 && token < a.tokens) ? token : 0) * a.row_stride * kSize;
  };
  auto open = [&](int i) {  // the row of entry i of this group
    row = __shfl_sync(0xffffffffu, now.y, i % 32);
    row_begin = __shfl_sync(0xffffffffu, now.z, i % 32);
    row_end = __shfl_sync(0xffffffffu, now.w, i % 32);
  };
  auto add = [&](int n, const Eight<kFp32, kVec, kCount>& raw) {
    float x[kCount];
    widen_eight<kFp32, kVec, kCount>(raw, x);
#pragma unroll
    for (int k = 0; k < kCount / 2; ++k) sum[n][k] = add2(sum[n][k], pair(x[2 * k], x[2 * k + 1]));
  };
  look();  // q is below 32: it lies within the run
  if constexpr (kVec == 8) {
    constexpr int kWords = 2;  // 16-byte words of a lane's row: of one part (fp32), of two
    extern __shared__ uint4 ring[];  // [warp][slot][word][lane]
    uint4* const mine = ring + threadIdx.x / 32 * kSumDepth * kWords * 32 + lane;
    const bool some[kWords] = {lane * 8 < cols, kFp32 ? lane * 8 < cols : lane * 8 + kPart < cols};
    const int word = kFp32 ? 16 : kPart * 2, step = lane * (kFp32 ? 32 : 16);  // bytes
    auto fetch = [&](int i, int slot) {
      if (i < end) {
        const char* of_i = row_at(i) + step;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
          if (some[w]) copy_async<16>(mine + (slot * kWords + w) * 32, of_i + w * word);
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kSumDepth; ++i) fetch(q + i, i);
    // rolled: the code of a row's end is long, and would stand here kSumDepth times
    int slot = 0;
#pragma unroll 1
    for (bool opens = true;; ++q, opens = false) {
      if (q == group + 32) {
        group += 32;
        now = next;
        next = third;
        look();
      }
      if (opens || q == end || (begins >> (q % 32) & 1u)) {
        if (!opens) put();
        if (q == end) break;
        open(q);
      }
      copy_wait<kSumDepth - 1>();
      uint4 u[kWords];
#pragma unroll
      for (int w = 0; w < kWords; ++w) u[w] = some[w] ? mine[(slot * kWords + w) * 32] : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (kFp32) {
        add(0, Eight<true, 8, 8>{{u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w}});
      } else {
#pragma unroll
        for (int w = 0; w < kWords; ++w) add(w, Eight<false, 8, 8>{{u[w].x, u[w].y, u[w].z, u[w].w}});
      }
      fetch(q + kSumDepth, slot);  // where this one was
      slot = (slot + 1) % kSumDepth;
    }
    copy_wait<0>();
  } else {
    constexpr int kRows = 4;  // in flight
    bool opens = true;
#pragma unroll 1
    for (; q < end; q += kRows) {
      Eight<kFp32, kVec, kCount> raw[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (q + i < end) load_eight<kFp32, kVec, kCount>(row_at(q + i), lane, 32, cols, &raw[i]);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int here = q + i;
        if (here >= end) break;
        if (here == group + 32) {
          group += 32;
          now = next;
          next = third;
          look();
        }
        if (opens || (begins >> (here % 32) & 1u)) {
          if (!opens) put();
          open(here);
        }
        opens = false;
        add(0, raw[i]);
      }
    }
    put();
  }
}

// A row in parts: four columns a lane, every warp a contiguous share of the
// parts, then warp after warp.
template <bool kOutFp32>
__global__ void __launch_bounds__(kJoinWarps * 32) embedding_join_kernel(const __grid_constant__ EmbArgs a) {
  __shared__ float4 sums[kJoinWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long items = static_cast<long long>(a.live[1]) * a.slabs;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int4 e = a.heavy[item / a.slabs];  // first run, row, parts: one of that run, then of those behind it
    if (!ZFS_CHECK(e.x >= 0 && e.z > 0 && e.z <= a.runs - e.x && e.y >= 0 && e.y < a.vocab)) continue;
    const int c = static_cast<int>(item % a.slabs) * 128 + lane * 4;
    const int share = (e.z + kJoinWarps - 1) / kJoinWarps, from = warp * share;
    const int to = from + share < e.z ? from + share : e.z;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < a.dim) {
#pragma unroll 8
      for (int p = from; p < to; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(a.parts + ((static_cast<long long>(e.x) + p) * 2 + (p == 0)) * a.pitch + c);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
      }
    }
    __syncthreads();
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kJoinWarps; ++w) {
        const float4 x = sums[w][lane];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
      }
      const float all[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (c + k >= a.dim) break;
        const long long o = e.y * a.out_stride + c + k;
        float x = all[k] * a.scale;
        if (a.accumulate) x += load_scalar(a.out, kOutFp32, o);
        store_scalar(a.out, kOutFp32, o, x);
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------
// The gradient's workspace (each part 16-byte aligned).
struct Workspace {
  long long sorted, counts, live, heavy, parts, total;
  int runs, pitch, chunk;
  long long heavy_rows;  // more tokens than that no rows can be in parts
};
// Long runs make few parts, short ones many warps: the longest that still gives
// every one of 152 SMs 32 warps (152 whatever the device: the workspace's size is
// asked for without one), counting warps of 256 columns, 64 below kNarrow: single
// elements, which the alignment may come to.  (bf16 of kNarrow to 2 kNarrow columns
// has four times as many; its best run is no other: 32768 tokens x 769 in runs of
// 8, 16, 32: 71, 66, 65 us, x 1001: 85, 77, 75, 8192 tokens x 1001: 27, 26, 29.)
constexpr int kRunWarps = 32 * 152;
int chunk_of(int64_t dim, int64_t tokens) {
  const int64_t width = dim < kNarrow ? kSumColumns<false, kFewSingles> : kSumColumns<false, kSingles>;
  const int64_t warps = (dim + width - 1) / width;
  int chunk = kMostChunk;
  while (chunk > kLeastChunk && tokens / chunk * warps < kRunWarps) chunk /= 2;
  return chunk;
}
Workspace lay_out(const zero_embedding_config& c, int64_t tokens) {
  Workspace w{};
  auto up = [](long long x) { return (x + 15) / 16 * 16; };
  w.chunk = chunk_of(c.dim, tokens);
  w.heavy_rows = tokens / (2 * w.chunk + 1);
  w.runs = static_cast<int>((tokens + w.chunk - 1) / w.chunk);
  w.pitch = static_cast<int>((c.dim + 3) / 4 * 4);
  w.counts = w.sorted + tokens * 16;
  w.live = w.counts + up(c.rows * 4);
  w.heavy = w.live + 16;
  w.parts = w.heavy + w.heavy_rows * 16;
  w.total = w.parts + (w.heavy_rows ? w.runs * 2LL * w.pitch * 4 : 0);
  return w;
}

// Sorting CTAs: more where the counters of their rows would not fit.
int remainders_of(int64_t rows) {
  int remainders = kSortCtas;
  while ((rows + remainders - 1) / remainders > kSortRows) remainders *= 2;
  return remainders;
}
// Every sorting CTA looks at every id: together 170 ids a nanosecond where they
// read them again (2^24 tokens, 2^20 rows: 103 ms), 1600 where lists hold their tokens
// (2^22, 2^22: 11 ms).  More looks than this would hold the GPU for many seconds.
constexpr int64_t kMostLooks = 1LL << 40;

zero_status check_embedding(const zero_embedding_config* c, int64_t tokens) {
  if (!c) return refuse(ZERO_EINVAL, "config is NULL");
  if (tokens < 0 || tokens > (1LL << 30)) return refuse(ZERO_EINVAL, "tokens not in 0..2^30");
  if (c->rows < 0 || c->rows > (1LL << 30)) return refuse(ZERO_EINVAL, "rows not in 0..2^30");
  if (c->dim < 1 || c->dim > (1 << 24)) return refuse(ZERO_EINVAL, "dim not in 1..2^24");
  if (!is_dtype(c->dtype)) return refuse(ZERO_EINVAL, "dtype is neither bf16 (0) nor fp32 (1)");
  if (c->id_bytes != 4 && c->id_bytes != 8) return refuse(ZERO_EINVAL, "ids must have 4 or 8 bytes");
  if (!std::isfinite(c->scale)) return refuse(ZERO_EINVAL, "scale must be finite");
  return ZERO_OK;
}

zero_status check_backward(const zero_embedding_config* c, int64_t tokens) {
  const zero_status st = check_embedding(c, tokens);
  if (st != ZERO_OK) return st;
  if (tokens > kMostLooks / remainders_of(c->rows)) return refuse(ZERO_EINVAL, "rows and tokens are too many together");
  return ZERO_OK;
}

zero_status check_rows(const void* p, int64_t stride, int dtype, const char* text) {
  if (misplaced(p, dtype_bytes(dtype)) || stride < 0) return refuse(ZERO_EINVAL, text);
  return ZERO_OK;
}

int lanes_of(const EmbArgs& a) {
  const int need = (a.dim + 7) / 8;
  return power_of_two(need < kEmbThreads ? need : kEmbThreads);
}

template <typename Id>
void launch_lookup(const EmbArgs& a, bool fp32, bool vec, dim3 grid, cudaStream_t s) {
  if (fp32) {
    if (vec) embedding_kernel<true, 8, Id><<<grid, kEmbThreads, 0, s>>>(a);
    else embedding_kernel<true, 1, Id><<<grid, kEmbThreads, 0, s>>>(a);
  } else {
    if (vec) embedding_kernel<false, 8, Id><<<grid, kEmbThreads, 0, s>>>(a);
    else embedding_kernel<false, 1, Id><<<grid, kEmbThreads, 0, s>>>(a);
  }
}
template <typename Id>
zero_status launch_sort(const EmbArgs& a, int shared, cudaStream_t s) {
  // beyond what every kernel may have
  if (shared > 12 * 1024 && allow_shared<embedding_sort_kernel<Id>, 160 * 1024>() != cudaSuccess)
    return launch_status("embedding sort's shared memory");
  embedding_sort_kernel<Id><<<a.remainders, kSortThreads, shared, s>>>(a);
  return launch_status("embedding sort launch");
}
template <bool kFp32, bool kOutFp32>
void launch_sum(const EmbArgs& a, int mode, dim3 grid, cudaStream_t s) {
  const dim3 block(kSumThreads);
  if (mode == kVectors) {
    if (allow_shared<embedding_sum_kernel<kFp32, kOutFp32, kVectors>, kSumShared>() != cudaSuccess) return;  // the launch's error
    launch_after(embedding_sum_kernel<kFp32, kOutFp32, kVectors>, grid, block, kSumShared, s, a);
  } else if (mode == kSingles) {
    launch_after(embedding_sum_kernel<kFp32, kOutFp32, kSingles>, grid, block, 0, s, a);
  } else {
    launch_after(embedding_sum_kernel<kFp32, kOutFp32, kFewSingles>, grid, block, 0, s, a);
  }
}

}  // namespace

unsigned int embedding_debug_failures() {
#ifdef ZFS_DEBUG_CHECKS
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_debug_failures, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
#else
  return 0;
#endif
}

}  // namespace zfs

extern "C" {

zero_status zero_embedding(const zero_embedding_config* cfg, int64_t tokens, const void* ids, const void* table,
                           int64_t table_stride, void* out, int64_t out_stride, void* stream) {
  using namespace zfs;
  zero_status st = check_embedding(cfg, tokens);
  if (st != ZERO_OK) return st;
  if (tokens == 0) return ZERO_OK;
  if (misplaced(ids, cfg->id_bytes)) return refuse(ZERO_EINVAL, "ids are NULL or misaligned");
  if (cfg->rows > 0 &&
      (st = check_rows(table, table_stride, cfg->dtype, "table is NULL or misaligned, or its stride negative")) != ZERO_OK)
    return st;
  if ((st = check_rows(out, out_stride, cfg->dtype, "out is NULL or misaligned, or its stride negative")) != ZERO_OK) return st;
  if (rows_overlap(out_stride, tokens, cfg->dim)) return refuse(ZERO_EINVAL, "out's stride makes its rows overlap");
  EmbArgs a{};
  a.tokens = tokens;
  a.vocab = static_cast<int>(cfg->rows);
  a.dim = static_cast<int>(cfg->dim);
  a.ids = ids;
  a.wide_ids = cfg->id_bytes == 8;
  a.rows = table;
  a.row_stride = table_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.scale = cfg->scale;
  a.lanes = lanes_of(a);
  const bool vec = a.dim % 8 == 0 && rows_aligned(table, table_stride, cfg->rows, cfg->dtype) &&
                   rows_aligned(out, out_stride, tokens, cfg->dtype);
  const long long per_cta = kEmbThreads / a.lanes, want = (tokens + per_cta - 1) / per_cta;
  const int slabs = (a.dim + a.lanes * 8 - 1) / (a.lanes * 8);
  const long long most = static_cast<long long>(sm_count()) * kLookupCtas;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), slabs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp32 = cfg->dtype == ZERO_GRAD_FP32;
  if (a.wide_ids) launch_lookup<long long>(a, fp32, vec, grid, s);
  else launch_lookup<int>(a, fp32, vec, grid, s);
  return launch_status("embedding launch");
}

zero_status zero_embedding_backward_workspace_bytes(const zero_embedding_config* cfg, int64_t tokens, int64_t* bytes) {
  if (!bytes) return zfs::refuse(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_backward(cfg, tokens);
  if (st != ZERO_OK) return st;
  *bytes = zfs::lay_out(*cfg, tokens).total;
  return ZERO_OK;
}

zero_status zero_embedding_backward(const zero_embedding_config* cfg, int64_t tokens, const void* ids, const void* dout,
                                    int64_t dout_stride, void* dtable, int32_t dtable_dtype, int64_t dtable_stride,
                                    int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  using namespace zfs;
  zero_status st = check_backward(cfg, tokens);
  if (st != ZERO_OK) return st;
  if (!is_dtype(dtable_dtype)) return refuse(ZERO_EINVAL, "dtable_dtype is neither bf16 (0) nor fp32 (1)");
  if (accumulate != 0 && accumulate != 1) return refuse(ZERO_EINVAL, "accumulate must be 0 or 1");
  if (cfg->rows == 0 || (accumulate && tokens == 0)) return ZERO_OK;
  if ((st = check_rows(dtable, dtable_stride, dtable_dtype, "dtable is NULL or misaligned, or its stride negative")) != ZERO_OK)
    return st;
  if (rows_overlap(dtable_stride, cfg->rows, cfg->dim)) return refuse(ZERO_EINVAL, "dtable's stride makes its rows overlap");
  if (tokens > 0) {
    if (misplaced(ids, cfg->id_bytes)) return refuse(ZERO_EINVAL, "ids are NULL or misaligned");
    if ((st = check_rows(dout, dout_stride, cfg->dtype, "dout is NULL or misaligned, or its stride negative")) != ZERO_OK)
      return st;
  }
  const Workspace w = lay_out(*cfg, tokens);
  if (misplaced(workspace, 16)) return refuse(ZERO_EINVAL, "workspace is NULL or not 16-byte aligned");
  if (workspace_bytes < w.total) return refuse(ZERO_EINVAL, "workspace is too small");
  char* at = static_cast<char*>(workspace);
  EmbArgs a{};
  a.tokens = tokens;
  a.vocab = static_cast<int>(cfg->rows);
  a.dim = static_cast<int>(cfg->dim);
  a.ids = ids;
  a.wide_ids = cfg->id_bytes == 8;
  a.rows = dout;
  a.row_stride = dout_stride;
  a.out = dtable;
  a.out_stride = dtable_stride;
  a.scale = cfg->scale;
  a.accumulate = accumulate;
  a.sorted = reinterpret_cast<int4*>(at + w.sorted);
  a.counts = reinterpret_cast<int*>(at + w.counts);
  a.live = reinterpret_cast<int*>(at + w.live);
  a.heavy = reinterpret_cast<int4*>(at + w.heavy);
  a.parts = reinterpret_cast<float*>(at + w.parts);
  a.pitch = w.pitch;
  a.runs = w.runs;
  a.chunk = w.chunk;
  a.slabs = (a.dim + 127) / 128;
  a.remainders = remainders_of(a.vocab);
  a.per_cta = (a.vocab + a.remainders - 1) / a.remainders;
  const int shared = (kSortWarps * a.per_cta + a.per_cta + 1) * static_cast<int>(sizeof(int));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp32 = cfg->dtype == ZERO_GRAD_FP32, out32 = dtable_dtype == ZERO_GRAD_FP32;
  const bool vec = a.dim % 8 == 0 && rows_aligned(dout, dout_stride, tokens, cfg->dtype) &&
                   rows_aligned(dtable, dtable_stride, cfg->rows, dtable_dtype);
  // unaligned rows, us with two single elements a lane | with eight:
  //   bf16, 4096 tokens x 769, 1001, 1301:  17, 18, 21 | 19, 19, 19;  32768 x 513, 1001:  46, 65 | 55, 68
  //   fp32, 4096 tokens x 449, 769, 1001:   15, 18, 19 | 19, 17, 18;  32768 x 257, 513:   40, 47 | 44, 40
  // (32768 x 1301 bf16 would gain, too: 76 | 96; the border does not look at the tokens)
  const int mode = vec ? kVectors : a.dim < (fp32 ? kNarrow : 2 * kNarrow) ? kFewSingles : kSingles;
  const int width = mode == kFewSingles ? kSumColumns<false, kFewSingles> : mode == kSingles || fp32 ? kSumColumns<true, kVectors> : kSumColumns<false, kVectors>;
  a.columns = (a.dim + width - 1) / width;
  const long long zeros = accumulate ? 0 : (a.vocab + 31LL) / 32, jobs = a.runs + zeros;
  if (jobs * a.columns / kSumWarps > INT32_MAX - 2) return refuse(ZERO_EINVAL, "tokens, rows and dim are too large together");
  st = a.wide_ids ? launch_sort<long long>(a, shared, s) : launch_sort<int>(a, shared, s);
  if (st != ZERO_OK) return st;
  const dim3 grid(ctas_of(a.runs, a.columns) + ctas_of(zeros, a.columns));
  if (grid.x > 0) {
    if (fp32) out32 ? launch_sum<true, true>(a, mode, grid, s) : launch_sum<true, false>(a, mode, grid, s);
    else out32 ? launch_sum<false, true>(a, mode, grid, s) : launch_sum<false, false>(a, mode, grid, s);
  }
  if ((st = launch_status("embedding sum launch")) != ZERO_OK) return st;
  if (w.heavy_rows > 0) {
    const long long items = w.heavy_rows * a.slabs, most = 4LL * sm_count();
    const dim3 ctas(static_cast<unsigned>(items < most ? items : most));
    if (out32) launch_after(embedding_join_kernel<true>, ctas, dim3(kJoinWarps * 32), 0, s, a);
    else launch_after(embedding_join_kernel<false>, ctas, dim3(kJoinWarps * 32), 0, s, a);
    st = launch_status("embedding join launch");
  }
  return st;
}

}  // extern "C"
