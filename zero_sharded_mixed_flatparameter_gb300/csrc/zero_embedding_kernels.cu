// Embedding lookup with a factor, and the table's gradient by sorted tokens;
// and their C calls.
//
//   out[t] = scale * table[id[t]]         (zeros where id[t] is no row)
//   dtable[v] = scale * sum of dout[t] over the tokens t with id[t] = v
//
// The gradient takes three launches.  The first sorts: every CTA owns a range
// of rows, reads all ids (they stay in L2), counts those before its range (so
// that it knows where its tokens go without asking another CTA) and places its
// own in the order of (row, token).  The second sums: a run of kChunk sorted
// tokens at a time, rows that lie in one run whole, the run's first and last
// row in part, and zeros for the rows without tokens.  The third joins the
// parts of a row in order.  Each sum has one order: the same call gives the
// same bits.

#include <cmath>

#include "zero_flatstep.h"
#include "zero_norm_internal.h"
#include "zero_rows.cuh"
#include "zero_rows_host.h"

namespace zfs {
namespace {

constexpr int kEmbThreads = 256;
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortRows = 1536;   // of a CTA at most: a counter for each and every warp, 192 KB
constexpr int kSortLoads = 8;     // ids in flight per lane
constexpr int kChunk = 32;        // sorted tokens of a run
constexpr int kZeroRows = 16;     // table rows of a CTA that writes zeros
constexpr int kJoinWarps = 8;

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
  int2* sorted;                // (token, row) in the order of (row, token)
  int* begin;                  // [vocab + 1] where a row's tokens begin in it
  int* crossing;               // how many runs end in the middle of a row's first part, then which
  float* parts;                // [run][part of the row before, of the last row][pitch]
  int pitch, per_cta;          // pitch: columns of a part, per_cta: table rows of a sorting CTA
  int runs, slabs;
};

// The row of token t, -1 if it has none.
__device__ __forceinline__ int row_of(const EmbArgs& a, long long t) {
  if (a.wide_ids) {
    const long long id = static_cast<const long long*>(a.ids)[t];
    return id >= 0 && id < a.vocab ? static_cast<int>(id) : -1;
  }
  const int id = static_cast<const int*>(a.ids)[t];
  return id >= 0 && id < a.vocab ? id : -1;
}

template <bool kFp32, int kVec>
__global__ void __launch_bounds__(kEmbThreads) embedding_kernel(const __grid_constant__ EmbArgs a) {
  constexpr int kRows = 4;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kEmbThreads / lanes;
  const long long step = static_cast<long long>(gridDim.x) * per_cta;
  const int at = blockIdx.y * lanes * 8, cols = a.dim - at;
  for (long long t0 = static_cast<long long>(blockIdx.x) * per_cta + threadIdx.x / lanes; t0 < a.tokens;
       t0 += step * kRows) {
    int row[kRows];
    Eight<kFp32, kVec> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) row[i] = t0 + step * i < a.tokens ? row_of(a, t0 + step * i) : -1;
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

// Calls f(token, row - first, lanes of the warp that call it now, those of them
// with the same row) for every token of the warp's share whose row lies in
// [first, first + count), in the order of the tokens; returns how many of this
// lane's tokens have a row before `first`.
template <typename F>
__device__ __forceinline__ int walk_tokens(const EmbArgs& a, int first, int count, F f) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long share = (a.tokens + kSortThreads - 1) / kSortThreads * 32;
  const long long end = (warp + 1) * share < a.tokens ? (warp + 1) * share : a.tokens;
  int before = 0;
  for (long long t0 = warp * share; t0 < end; t0 += 32 * kSortLoads) {
    int row[kSortLoads];
#pragma unroll
    for (int u = 0; u < kSortLoads; ++u) row[u] = t0 + 32 * u + lane < end ? row_of(a, t0 + 32 * u + lane) : -1;
#pragma unroll
    for (int u = 0; u < kSortLoads; ++u) {
      const int r = row[u] - first;
      before += row[u] >= 0 && r < 0;
      const bool in = row[u] >= 0 && r >= 0 && r < count;
      const unsigned some = __ballot_sync(0xffffffffu, in);
      if (some == 0u) continue;
      if (in) {
        f(static_cast<int>(t0 + 32 * u + lane), r, some, __match_any_sync(some, r));
      }
      __syncwarp();
    }
  }
  return before;
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ EmbArgs a) {
  extern __shared__ int counters[];  // [warp][row]
  __shared__ int sums[kSortWarps];
  __shared__ int base;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned lower = (1u << lane) - 1u;  // the lanes before this one
  const int first = blockIdx.x * a.per_cta;
  const int count = a.vocab - first < a.per_cta ? a.vocab - first : a.per_cta;
  int* mine = counters + warp * a.per_cta;
  for (int i = threadIdx.x; i < kSortWarps * a.per_cta; i += kSortThreads) counters[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.crossing[0] = 0;
  __syncthreads();
  int before = walk_tokens(a, first, count, [&](int, int r, unsigned, unsigned same) {
    if ((same & lower) == 0u) mine[r] += __popc(same);
  });
  before = warp_total(before);
  if (lane == 0) sums[warp] = before;
  __syncthreads();
  if (warp == 0) {
    before = warp_total(sums[lane]);
    if (lane == 0) base = before;
  }
  __syncthreads();
  // where every (row, warp) begins: over the rows kSortThreads at a time
  int running = base;
  for (int r0 = 0; r0 < count; r0 += kSortThreads) {
    const int r = r0 + threadIdx.x;
    int total = 0;
    if (r < count) {
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
    __syncthreads();
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int before_mine = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before_mine += sums[w];
      all += sums[w];
    }
    if (r < count) {
      const int at = running + before_mine + scan - total;
      a.begin[first + r] = at;
      for (int w = 0; w < kSortWarps; ++w) counters[w * a.per_cta + r] += at;
    }
    running += all;
  }
  if (first + count == a.vocab && threadIdx.x == 0) a.begin[a.vocab] = running;
  if (running == base) return;
  __syncthreads();
  walk_tokens(a, first, count, [&](int t, int r, unsigned some, unsigned same) {
    const int at = mine[r];
    __syncwarp(some);
    if ((same & lower) == 0u) mine[r] = at + __popc(same);
    const int to = at + __popc(same & lower);
    if (ZFS_CHECK(to >= 0 && to < a.tokens)) a.sorted[to] = make_int2(t, first + r);
  });
}

// A thread's eight columns of the table's gradient.
template <bool kFp32, int kVec>
__device__ __forceinline__ void put_row(const EmbArgs& a, int row, int at, int lane, int lanes, const float* sum) {
  constexpr long long kSize = kFp32 ? 4 : 2;
  char* to = static_cast<char*>(a.out) + (row * a.out_stride + at) * kSize;
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = sum[k] * a.scale;
  if (a.accumulate) {
    Eight<kFp32, kVec> old;
    float y[8];
    load_eight<kFp32, kVec>(to, lane, lanes, a.dim - at, &old);
    widen_eight<kFp32, kVec>(old, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += y[k];
  }
  store_eight<kFp32, kVec>(to, lane, lanes, a.dim - at, x);
}

template <bool kFp32, bool kOutFp32, int kVec>
__global__ void __launch_bounds__(kEmbThreads) embedding_sum_kernel(const __grid_constant__ EmbArgs a, int run_ctas) {
  constexpr int kRows = 8;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kEmbThreads / lanes;
  const int at = blockIdx.y * lanes * 8, cols = a.dim - at;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) >= run_ctas) {
    const float zero[8] = {};
    const int v0 = (blockIdx.x - run_ctas) * kZeroRows;
    for (int i = threadIdx.x / lanes; i < kZeroRows; i += per_cta) {
      const int v = v0 + i;
      if (v < a.vocab && a.begin[v] == a.begin[v + 1])
        store_eight<kOutFp32, kVec>(static_cast<char*>(a.out) + (v * a.out_stride + at) * (kOutFp32 ? 4 : 2), lane, lanes,
                                    cols, zero);
    }
    return;
  }
  const int live = a.begin[a.vocab];
  const long long run = static_cast<long long>(blockIdx.x) * per_cta + threadIdx.x / lanes;
  const long long begin = run * kChunk;
  if (begin >= live) return;
  const int end = begin + kChunk < live ? static_cast<int>(begin) + kChunk : live;
  int row = a.sorted[begin].y;
  // a row that began before this run, or goes on after it, is summed in part
  bool head = begin > 0 && a.sorted[begin - 1].y == row;
  const bool open = end < live && a.sorted[end].y == a.sorted[end - 1].y;
  float sum[8] = {};
  auto put = [&](bool last) {
    if (head || (last && open)) {
      float* to = a.parts + (run * 2 + (head ? 0 : 1)) * a.pitch + at;
      if (!head && lane == 0 && blockIdx.y == 0) a.crossing[1 + atomicAdd(a.crossing, 1)] = static_cast<int>(run);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = column<kVec>(k, lane, lanes);
        if (c < cols) to[c] = sum[k];
      }
    } else {
      put_row<kOutFp32, kVec>(a, row, at, lane, lanes, sum);
    }
    head = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
  };
  for (int p = static_cast<int>(begin); p < end; p += kRows) {
    int2 entry[kRows];
    Eight<kFp32, kVec> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) entry[i] = p + i < end ? a.sorted[p + i] : make_int2(0, -1);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      load_eight<kFp32, kVec>(static_cast<const char*>(a.rows) + (entry[i].x * a.row_stride + at) * kSize, lane, lanes,
                              entry[i].y >= 0 ? cols : 0, &raw[i]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (p + i >= end) break;
      if (entry[i].y != row) {
        put(false);
        row = entry[i].y;
      }
      float x[8];
      widen_eight<kFp32, kVec>(raw[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += x[k];
    }
  }
  put(true);
}

// A row whose tokens lie in several runs: four columns a lane, every warp a
// contiguous share of the parts, then warp after warp.
template <bool kOutFp32>
__global__ void __launch_bounds__(kJoinWarps * 32) embedding_join_kernel(const __grid_constant__ EmbArgs a) {
  __shared__ float4 sums[kJoinWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long items = static_cast<long long>(a.crossing[0]) * a.slabs;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int run = a.crossing[1 + item / a.slabs], c = static_cast<int>(item % a.slabs) * 128 + lane * 4;
    const int row = a.sorted[static_cast<long long>(run) * kChunk + kChunk - 1].y;
    const int parts = (a.begin[row + 1] - 1) / kChunk - run + 1;  // one of this run, then of those behind it
    const int share = (parts + kJoinWarps - 1) / kJoinWarps, from = warp * share;
    const int to = from + share < parts ? from + share : parts;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < a.dim) {
#pragma unroll 8
      for (int p = from; p < to; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(a.parts + ((static_cast<long long>(run) + p) * 2 + (p == 0)) * a.pitch + c);
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
        const long long o = row * a.out_stride + c + k;
        float x = all[k] * a.scale;
        if (a.accumulate) x += load_scalar(a.out, kOutFp32, o);
        store_scalar(a.out, kOutFp32, o, x);
      }
    }
  }
}

// ---- host ----------------------------------------------------------------------
// The gradient's workspace: sorted tokens, rows' beginnings, list of rows in
// parts, the parts (each 16-byte aligned).
struct Workspace {
  long long sorted, begin, crossing, parts, total;
  int runs, pitch;
};
Workspace lay_out(const zero_embedding_config& c, int64_t tokens) {
  Workspace w{};
  auto up = [](long long x) { return (x + 15) / 16 * 16; };
  w.runs = static_cast<int>((tokens + kChunk - 1) / kChunk);
  w.pitch = static_cast<int>((c.dim + 3) / 4 * 4);
  w.sorted = 0;
  w.begin = up(tokens * 8);
  w.crossing = w.begin + up((c.rows + 1) * 4);
  w.parts = w.crossing + up((w.runs + 1LL) * 4);
  w.total = w.parts + (w.runs > 1 ? w.runs * 2LL * w.pitch * 4 : 0);
  return w;
}

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

zero_status check_rows(const void* p, int64_t stride, int dtype, const char* text) {
  if (misplaced(p, dtype_bytes(dtype)) || stride < 0) return refuse(ZERO_EINVAL, text);
  return ZERO_OK;
}

int lanes_of(const EmbArgs& a) {
  const int need = (a.dim + 7) / 8;
  return power_of_two(need < kEmbThreads ? need : kEmbThreads);
}

template <bool kFp32, bool kOutFp32>
void launch_sum(const EmbArgs& a, bool vec, dim3 grid, int run_ctas, cudaStream_t s) {
  if (vec) launch_after(embedding_sum_kernel<kFp32, kOutFp32, 8>, grid, dim3(kEmbThreads), 0, s, a, run_ctas);
  else launch_after(embedding_sum_kernel<kFp32, kOutFp32, 1>, grid, dim3(kEmbThreads), 0, s, a, run_ctas);
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
  const long long most = static_cast<long long>(sm_count()) * (2048 / kEmbThreads);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), slabs);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->dtype == ZERO_GRAD_FP32) {
    if (vec) embedding_kernel<true, 8><<<grid, kEmbThreads, 0, s>>>(a);
    else embedding_kernel<true, 1><<<grid, kEmbThreads, 0, s>>>(a);
  } else {
    if (vec) embedding_kernel<false, 8><<<grid, kEmbThreads, 0, s>>>(a);
    else embedding_kernel<false, 1><<<grid, kEmbThreads, 0, s>>>(a);
  }
  return launch_status("embedding launch");
}

zero_status zero_embedding_backward_workspace_bytes(const zero_embedding_config* cfg, int64_t tokens, int64_t* bytes) {
  if (!bytes) return zfs::refuse(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_embedding(cfg, tokens);
  if (st != ZERO_OK) return st;
  *bytes = zfs::lay_out(*cfg, tokens).total;
  return ZERO_OK;
}

zero_status zero_embedding_backward(const zero_embedding_config* cfg, int64_t tokens, const void* ids, const void* dout,
                                    int64_t dout_stride, void* dtable, int32_t dtable_dtype, int64_t dtable_stride,
                                    int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  using namespace zfs;
  zero_status st = check_embedding(cfg, tokens);
  if (st != ZERO_OK) return st;
  if (!is_dtype(dtable_dtype)) return refuse(ZERO_EINVAL, "dtable_dtype is neither bf16 (0) nor fp32 (1)");
  if (accumulate != 0 && accumulate != 1) return refuse(ZERO_EINVAL, "accumulate must be 0 or 1");
  if (cfg->rows == 0 || (accumulate && tokens == 0)) return ZERO_OK;
  if ((st = check_rows(dtable, dtable_stride, dtable_dtype, "dtable is NULL or misaligned, or its stride negative")) != ZERO_OK)
    return st;
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
  a.sorted = reinterpret_cast<int2*>(at + w.sorted);
  a.begin = reinterpret_cast<int*>(at + w.begin);
  a.crossing = reinterpret_cast<int*>(at + w.crossing);
  a.parts = reinterpret_cast<float*>(at + w.parts);
  a.pitch = w.pitch;
  a.runs = w.runs;
  a.slabs = (a.dim + 127) / 128;
  a.lanes = lanes_of(a);
  // a CTA of sorting per SM, more where its rows' counters would not fit
  a.per_cta = (a.vocab + sm_count() - 1) / sm_count();
  if (a.per_cta > kSortRows) a.per_cta = kSortRows;
  const int sorting = (a.vocab + a.per_cta - 1) / a.per_cta;
  const size_t counters = static_cast<size_t>(kSortWarps) * a.per_cta * sizeof(int);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // beyond what every kernel may have; set anew each time, as it belongs to the current context
  if (counters > 48 * 1024 - 1024 &&
      cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSortWarps * kSortRows * sizeof(int))) != cudaSuccess)
    return launch_status("embedding sort's shared memory");
  embedding_sort_kernel<<<sorting, kSortThreads, counters, s>>>(a);
  if ((st = launch_status("embedding sort launch")) != ZERO_OK) return st;
  const bool fp32 = cfg->dtype == ZERO_GRAD_FP32, out32 = dtable_dtype == ZERO_GRAD_FP32;
  const bool vec = a.dim % 8 == 0 && rows_aligned(dout, dout_stride, tokens, cfg->dtype) &&
                   rows_aligned(dtable, dtable_stride, cfg->rows, dtable_dtype);
  const int per_cta = kEmbThreads / a.lanes, run_ctas = (a.runs + per_cta - 1) / per_cta;
  const int zero_ctas = accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
  const dim3 grid(run_ctas + zero_ctas, (a.dim + a.lanes * 8 - 1) / (a.lanes * 8));
  if (fp32) out32 ? launch_sum<true, true>(a, vec, grid, run_ctas, s) : launch_sum<true, false>(a, vec, grid, run_ctas, s);
  else out32 ? launch_sum<false, true>(a, vec, grid, run_ctas, s) : launch_sum<false, false>(a, vec, grid, run_ctas, s);
  if ((st = launch_status("embedding sum launch")) != ZERO_OK) return st;
  if (a.runs > 1) {  // one run has no row in parts
    const long long items = static_cast<long long>(a.runs) * a.slabs, most = 8LL * sm_count();
    const dim3 ctas(static_cast<unsigned>(items < most ? items : most));
    if (out32) launch_after(embedding_join_kernel<true>, ctas, dim3(kJoinWarps * 32), 0, s, a);
    else launch_after(embedding_join_kernel<false>, ctas, dim3(kJoinWarps * 32), 0, s, a);
    st = launch_status("embedding join launch");
  }
  return st;
}

}  // extern "C"
