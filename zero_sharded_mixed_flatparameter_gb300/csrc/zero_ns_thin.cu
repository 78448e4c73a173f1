// Newton-Schulz orthogonalisation of thin matrices, smaller side m <= kThin:
// the whole chain in one launch, a cluster of CTAs per matrix.
//
// Every step's factor is a polynomial of the same Gram matrix, so a few steps
// can run on m x m matrices alone and touch X twice:
//   A = X X^T;  per step P = a I + b A + c A A,  Q <- P Q,  A <- P (A P)
//   X <- Q X
// The rounding of A then grows by up to a^2 (11.9) a step instead of a: the
// products keep 22 bits (every operand is an fp16 pair hi + lo, a product is
// lo hi + hi lo + hi hi with fp32 sums that the tensor cores truncate: 1e-6)
// and two steps share a Gram matrix.  A rank-1 128 x 128 matrix is then 1.2e-5
// off after two steps, 1.4e-4 after three and 5.5e-2 after all five from one
// Gram matrix; restarted every two, 5e-4 after five.
//
// What bounds it is latency: each product of 128 takes under a microsecond,
// and the next one waits for it.  Hence one launch, operands that stay in
// shared memory (A, P, Q: 3 x 64 KB), and the columns of X split over up to 8
// CTAs whose partial Gram matrices are joined in distributed shared memory;
// every CTA then solves the chain by itself rather than wait for another.
// In the Muon step the momentum pass is the first thing the kernel does.

#include "zero_device.cuh"
#include "zero_muon_internal.h"
#include "zero_tensor.cuh"

namespace zfs {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSlice = 128;                        // columns of X at a time
constexpr uint32_t kBlockBytes = 128 * 128;        // 128 rows of 64 fp16, swizzled
constexpr uint32_t kHalfBytes = 2 * kBlockBytes;   // 128 x 128 fp16
constexpr uint32_t kPairBytes = 2 * kHalfBytes;    // hi and lo
constexpr uint32_t kSmemBytes = 3 * kPairBytes + 1024;
constexpr uint32_t kTmemColumns = 256;

struct Shared {
  uint64_t bar[3];
  double sum;  // of this CTA's columns, read by the cluster
  float warp_sum[kWarps];
  float norm_scale;
  uint32_t tmem;
  int gave_up;
};

// ---- shared-memory pairs -----------------------------------------------------
// Address of the 8-element chunk `chunk` (of 16) of row r in a 128 x 128 half.
__device__ __forceinline__ uint32_t chunk_at(uint32_t half, int r, int chunk) {
  return half + (chunk / 8) * kBlockBytes + r * 128 + (((chunk % 8) ^ (r & 7)) << 4);
}
// The nearest fp16 pair of eight values.
__device__ __forceinline__ void split8(const float* x, uint32_t* hi, uint32_t* lo) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    hi[k] = half2_bits(x[2 * k], x[2 * k + 1]);
    const float2 h = half2_values(hi[k]);
    lo[k] = half2_bits(x[2 * k] - h.x, x[2 * k + 1] - h.y);
  }
}
__device__ __forceinline__ void store_pair(uint32_t buffer, int r, int chunk, const float* x) {
  uint32_t hi[4], lo[4];
  split8(x, hi, lo);
  sts16(chunk_at(buffer, r, chunk), make_uint4(hi[0], hi[1], hi[2], hi[3]));
  sts16(chunk_at(buffer + kHalfBytes, r, chunk), make_uint4(lo[0], lo[1], lo[2], lo[3]));
}
__device__ __forceinline__ void load_pair(uint32_t buffer, int r, int chunk, float* x) {
  const uint4 h = lds16(chunk_at(buffer, r, chunk)), l = lds16(chunk_at(buffer + kHalfBytes, r, chunk));
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 u = half2_values(hw[k]), v = half2_values(lw[k]);
    x[2 * k] = u.x + v.x;
    x[2 * k + 1] = u.y + v.y;
  }
}

// acc (128 rows, `n` columns) = sum over k < depth of the pair product of two
// buffers, A K-major and B K-major or MN-major.  One thread.
__device__ __forceinline__ void issue_pair(uint32_t acc, uint32_t a, uint32_t b, bool b_k_major, int n, int depth,
                                           bool accumulate) {
  const uint32_t idesc = (1u << 4) | (b_k_major ? 0u : 1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
  uint32_t on = accumulate ? 1 : 0;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {  // hi lo, lo hi, hi hi: the small terms first, as sums are truncated
    const uint32_t pa = a + (part == 1 ? kHalfBytes : 0), pb = b + (part == 0 ? kHalfBytes : 0);
#pragma unroll 1
    for (int k = 0; k < depth; k += 16) {
      const uint32_t ka = pa + (k / 64) * kBlockBytes + (k % 64) * 2;
      const uint32_t kb = b_k_major ? pb + (k / 64) * kBlockBytes + (k % 64) * 2 : pb + k * 128;
      mma<1>(acc, smem_desc(ka, true, 0), smem_desc(kb, b_k_major, kBlockBytes), idesc, on);
      on = 1;
    }
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t at) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// ---- the input ---------------------------------------------------------------
// A run of up to 8 contiguous elements of the matrix: X rows are the smaller
// side, so for a tall matrix a run holds consecutive rows of one X column.
struct Run {
  long long at;  // row-major index in the given orientation
  int row, col;  // of X, of the run's first element
  int count;     // elements that exist
};

struct Matrix {
  long long ld;  // elements between rows of the given orientation
  int m, n, mk;  // X is m x n; mk: m rounded up to 16
  bool tall;
};

// The i-th run of a slice, i < slice_runs(): lanes take consecutive chunks of
// a row (wide), or consecutive columns of X, one memory row each (tall).
__device__ __forceinline__ int slice_runs(const Matrix& x) { return x.mk * (kSlice / 8); }
__device__ __forceinline__ Run slice_run(const Matrix& x, int j0, int i) {
  Run r;
  if (x.tall) {
    r.row = i / kSlice * 8;
    r.col = j0 + i % kSlice;
    r.at = r.col * x.ld + r.row;
    r.count = r.col < x.n ? max(0, min(8, x.m - r.row)) : 0;
  } else {
    r.row = i / (kSlice / 8);
    r.col = j0 + i % (kSlice / 8) * 8;
    r.at = r.row * x.ld + r.col;
    r.count = r.row < x.m ? max(0, min(8, x.n - r.col)) : 0;
  }
  return r;
}

template <bool kFp32>
__device__ __forceinline__ void load_run(const void* base, const Run& r, bool vec, float* x) {
  if (vec && r.count == 8) load8<kFp32, true>(base, r.at, 8, x);
  else load8<kFp32, false>(base, r.at, r.count, x);
}

// A slice of X0 as pairs in `buffer`; what does not exist is zero.
template <bool kFp32>
__device__ __forceinline__ void load_slice(const Matrix& x, const void* base, bool vec, int j0, float scale,
                                           uint32_t buffer) {
#pragma unroll 2
  for (int i = threadIdx.x; i < slice_runs(x); i += kThreads) {
    const Run r = slice_run(x, j0, i);
    float v[8];
    load_run<kFp32>(base, r, vec, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= scale;
    if (!x.tall) {
      store_pair(buffer, r.row, (r.col - j0) / 8, v);
    } else {
      uint32_t hi[4], lo[4];
      split8(v, hi, lo);
      const int c = r.col - j0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = chunk_at(buffer, r.row + k, c / 8) + c % 8 * 2;
        sts2(at, static_cast<uint16_t>(hi[k / 2] >> (16 * (k % 2))));
        sts2(at + kHalfBytes, static_cast<uint16_t>(lo[k / 2] >> (16 * (k % 2))));
      }
    }
  }
}

// The momentum pass over a slice: returns the thread's sum of squares.
template <bool kFp32>
__device__ __forceinline__ float momentum_slice(const ThinArgs& a, int mat, const Matrix& x, bool vec, int j0,
                                                float* update, unsigned* nf) {
  const float clip = a.clip ? *a.clip : 1.0f;
  const long long base = a.offset[mat];
  float sq = 0.0f;
  for (int i = threadIdx.x; i < slice_runs(x); i += kThreads) {
    const Run r = slice_run(x, j0, i);
    if (r.count == 0 || !ZFS_CHECK(base >= 0 && base + r.at + r.count <= a.total_padded)) continue;
    float g[8], y[8], m[8];
    load_run<kFp32>(a.g[mat][0], r, vec, g);
#pragma unroll 4
    for (int q = 1; q < a.n_ranks; ++q) {
      load_run<kFp32>(a.g[mat][q], r, vec, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = __fadd_rn(g[k], y[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = __fmul_rn(g[k], a.inv_n);
    *nf += tally_nonfinite<8>(g);
    load_run<true>(a.mom + base, r, vec, m);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (a.clip) g[k] = __fmul_rn(g[k], clip);
      m[k] = __fadd_rn(__fmul_rn(a.mu, m[k]), g[k]);
      y[k] = a.nesterov ? __fadd_rn(g[k], __fmul_rn(a.mu, m[k])) : m[k];
      sq += y[k] * y[k];
    }
    float* mom = a.mom + base + r.at;
    if (vec && r.count == 8) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        reinterpret_cast<float4*>(mom)[q] = make_float4(m[4 * q], m[4 * q + 1], m[4 * q + 2], m[4 * q + 3]);
        reinterpret_cast<float4*>(update + r.at)[q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < r.count) {
          mom[k] = m[k];
          update[r.at + k] = y[k];
        }
      }
    }
  }
  return sq;
}

// ---- the output --------------------------------------------------------------
// Eight consecutive X columns j .. j+7 of row i, finished values.
template <bool kMuon>
__device__ __forceinline__ void store_result(const ThinArgs& a, int mat, const Matrix& x, bool vec, int i, int j,
                                             float* y) {
  if (i >= x.m || j >= x.n) return;
  const int count = min(8, x.n - j);
  const long long ld = kMuon ? x.ld : a.out_row_stride;
  const long long at = x.tall ? j * ld + i : i * ld + j, next = x.tall ? ld : 1;
  if constexpr (kMuon) {
    const long long base = a.offset[mat] + at;
    if (!ZFS_CHECK(base >= 0 && base + (count - 1) * next < a.total_padded)) return;
    float* w = a.master + base;
    uint16_t* p = a.p16 + base;
    const float step = a.step[mat];
    if (vec && !x.tall && count == 8) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 old = reinterpret_cast<const float4*>(w)[q];
        const float o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[4 * q + k] = __fadd_rn(__fmul_rn(o[k], a.decay), __fmul_rn(-step, y[4 * q + k]));
        reinterpret_cast<float4*>(w)[q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < count) {
          const float z = __fadd_rn(__fmul_rn(w[k * next], a.decay), __fmul_rn(-step, y[k]));
          w[k * next] = z;
          p[k * next] = to_bf16_bits(z);
        }
      }
    }
  } else {
    uint16_t* d = a.out + mat * a.out_mat_stride + at;
    if (a.vec_out && !x.tall && count == 8) {
      *reinterpret_cast<uint4*>(d) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < count) d[k * next] = to_bf16_bits(y[k]);
    }
  }
}

// The same of an iterate between two Gram matrices, to the fp32 buffer.
__device__ __forceinline__ void store_iterate(const Matrix& x, float* to, int i, int j, const float* y) {
  if (i >= x.m || j >= x.n) return;
  const int count = min(8, x.n - j);
  float* d = to + (x.tall ? j * x.ld + i : i * x.ld + j);
  const long long next = x.tall ? x.ld : 1;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < count) d[k * next] = y[k];
}

// ---- the kernel --------------------------------------------------------------
// kCtas CTAs per matrix.  Every CTA of a cluster reaches every cluster barrier;
// one whose wait gave up (alive = false) only skips its work.
template <int kCtas, bool kMuon, bool kFp32>
__global__ void __launch_bounds__(kThreads, 1) ns_thin_kernel(const __grid_constant__ ThinArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sh;
  if constexpr (kMuon) {
    if (a.dev_t && *a.dev_t >= a.dev_steps) return;  // the same for the whole grid
  }
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = kCtas > 1 ? cluster_rank() : 0;
  const int mat = blockIdx.x / kCtas;
  const uint32_t b0 = (smem_u32(smem_raw) + 1023) & ~1023u, b1 = b0 + kPairBytes, b2 = b1 + kPairBytes;
  Matrix x;
  {
    const int at = kMuon ? mat : 0, rows = a.rows[at], cols = a.cols[at];
    x.tall = rows > cols;
    x.m = min(rows, cols);
    x.n = max(rows, cols);
    x.mk = (x.m + 15) / 16 * 16;
    x.ld = kMuon ? cols : a.src.row_stride;
  }
  const bool vec = kMuon ? (a.vec[mat / 32] >> (mat % 32)) & 1 : a.src.vec_ok != 0;
  // the Muon step's update, and the iterate between Gram matrices, row after row
  float* work = a.work + (kMuon ? a.work_offset[mat] : mat * a.work_mat_stride);
  Matrix xw = x;
  xw.ld = x.tall ? x.m : x.n;
  const bool vec_work = xw.ld % 8 == 0;
  const void* source = kMuon ? static_cast<const void*>(work)
                             : static_cast<const char*>(a.src.data) + mat * a.src.mat_stride * (kFp32 ? 4 : 2);
  if (tid == 0) {
    sh.gave_up = 0;
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&sh.bar[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc<1>(smem_u32(&sh.tmem), kTmemColumns);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sh.tmem;
  bool alive = true;
  uint32_t phase[3] = {0, 0, 0};
  // Waits for the products committed to barrier `i`; all threads.
  auto wait = [&](int i) {
    const bool ok = alive && wait_phase(smem_u32(&sh.bar[i]), phase[i], &sh.gave_up);
    phase[i] ^= 1;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    return ok;
  };
  // Makes shared-memory operands and drained accumulators ready for products.
  auto ready = [&](bool ok) {
    asm volatile("fence.proxy.async;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    alive = __syncthreads_and(ok ? 1 : 0) != 0;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  };

  // ---- norm (and momentum) over this CTA's slices ------------------------------
  float sq = 0.0f;
  unsigned nf = 0;
  for (int j0 = rank * kSlice; j0 < x.n; j0 += kCtas * kSlice) {
    if constexpr (kMuon) {
      sq += a.grad_fp32 ? momentum_slice<true>(a, mat, x, vec, j0, work, &nf)
                        : momentum_slice<false>(a, mat, x, vec, j0, work, &nf);
    } else {
      for (int i = tid; i < slice_runs(x); i += kThreads) {
        float v[8];
        load_run<kFp32>(source, slice_run(x, j0, i), vec, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sq += v[k] * v[k];
      }
    }
  }
  if constexpr (kMuon) flush_nonfinite(a.nonfinite, nf);
  // fp32 over a warp, fp64 above, by one thread (the GPU has few fp64 units)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0) sh.warp_sum[warp] = sq;
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < kWarps; ++w) t += sh.warp_sum[w];
    sh.sum = t;
  }
  if constexpr (kCtas > 1) cluster_sync();
  if (tid == 0) {
    double t = 0.0;
    if constexpr (kCtas > 1) {
      for (int r = 0; r < kCtas; ++r) t += ld_cluster_f64(map_rank(smem_u32(&sh.sum), r));
    } else {
      t = sh.sum;
    }
    sh.norm_scale = static_cast<float>(1.0 / (sqrt(t) + static_cast<double>(a.eps)));
  }
  __syncthreads();
  const float norm_scale = sh.norm_scale;
  const int mk = x.mk;
  // the epilogue's share of a thread: row `row`, a quarter of the columns
  const int row = (warp % 4) * 32 + lane, quarter = warp / 4;
  const bool in_rows = (warp % 4) * 32 < mk;  // the same for the whole warp
  const uint32_t tmem_row = tmem + (((warp % 4) * 32) << 16);
  auto product = [&](uint32_t acc, uint32_t p, uint32_t q) { issue_pair(acc, p, q, true, mk, mk, false); };
  auto go = [&](int i) { mma_commit<1>(smem_u32(&sh.bar[i])); };

  for (int begin = 0; begin < a.steps; begin += kThinChain) {
  const int end = min(begin + kThinChain, a.steps);
  const ThinStep& f0 = a.step_factors[begin];
  auto fetch = [&](int j0, uint32_t buffer) {
    if (begin == 0) load_slice<kFp32>(x, source, vec, j0, norm_scale * f0.x, buffer);
    else load_slice<true>(xw, work, vec_work, j0, f0.x, buffer);
  };

  // ---- Gram matrix: slices of X through the two buffers -------------------------
  int used = 0;
  bool ok = alive;
  for (int j0 = rank * kSlice; j0 < x.n; j0 += kCtas * kSlice, ++used) {
    const int i = used & 1;
    ok = alive;
    if (used >= 2) ok = wait(i);
    fetch(j0, i ? b1 : b0);
    ready(ok);
    if (tid == 0 && alive) {
      issue_pair(tmem, i ? b1 : b0, i ? b1 : b0, true, mk, kSlice, used > 0);
      mma_commit<1>(smem_u32(&sh.bar[i]));
    }
  }
  ok = alive;
  if (used >= 2) ok = wait(used & 1) && ok;
  if (used >= 1) ok = wait((used + 1) & 1) && ok;
  const float from_x = f0.gram;
  if constexpr (kCtas == 1) {
    // A straight from the accumulator
    if (ok && in_rows) {
      for (int c = quarter * 32; c < min(mk, quarter * 32 + 32); c += 16) {
        float y[16];
        __syncwarp();
        tmem_load16(tmem_row + c, y);
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] *= from_x;
        store_pair(b0, row, c / 8, y);
        store_pair(b0, row, c / 8 + 1, y + 8);
      }
    }
  } else {
    // Partial sums to this CTA's b2 (column after column: A is symmetric, and
    // lanes are rows); each CTA joins mk / kCtas columns in rank order and
    // gives them to all.
    if (ok && in_rows) {
      for (int c = quarter * 32; c < min(mk, quarter * 32 + 32); c += 16) {
        float y[16];
        __syncwarp();
        tmem_load16(tmem_row + c, y);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(b2 + ((c + k) * 128 + row) * 4),
                       "f"(used > 0 ? y[k] * from_x : 0.0f)
                       : "memory");
      }
    }
    cluster_sync();
    const int columns = mk / kCtas, first = rank * columns;
    for (int e = tid; e < columns * (mk / 2); e += kThreads) {
      const int c = first + e / (mk / 2), r = e % (mk / 2) * 2;
      float u = 0.0f, v = 0.0f;
#pragma unroll
      for (int q = 0; q < kCtas; ++q) {
        const uint32_t at = map_rank(b2 + (c * 128 + r) * 4, q);
        u += ld_cluster(at);
        v += ld_cluster(at + 4);
      }
      const uint32_t hi = half2_bits(u, v);
      const float2 h = half2_values(hi);
      const uint32_t lo = half2_bits(u - h.x, v - h.y);
      const uint32_t at = chunk_at(b0, c, r / 8) + r % 8 * 2;  // row c of A, columns r and r + 1
#pragma unroll
      for (int q = 0; q < kCtas; ++q) {
        st_cluster(map_rank(at, q), hi);
        st_cluster(map_rank(at + kHalfBytes, q), lo);
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    cluster_sync();
  }
  ready(ok);

  // ---- the chain on m x m matrices ----------------------------------------------
  // A in b0, P in b1, Q in b2; every matrix commutes with every other.
  for (int k = begin; k < end; ++k) {
    const bool first = k == begin, last = k + 1 == end;
    const ThinStep& f = a.step_factors[k];
    if (tid == 0 && alive) {
      product(tmem, b0, b0);  // A A
      go(0);
    }
    ok = wait(0);
    if (ok && in_rows) {
      const float fc = f.square, fb = f.gram_term, fa = f.identity;
      for (int c = quarter * 32; c < min(mk, quarter * 32 + 32); c += 16) {
        float y[16];
        __syncwarp();
        tmem_load16(tmem_row + c, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float old[8], z[8];
          load_pair(b0, row, c / 8 + h, old);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int col = c + 8 * h + q;
            z[q] = fmaf(fc, y[8 * h + q], fb * old[q]) + (col == row && row < x.m ? fa : 0.0f);
          }
          store_pair(b1, row, c / 8 + h, z);
          if (first) store_pair(b2, row, c / 8 + h, z);
        }
      }
    }
    ready(ok);
    if (first && last) break;
    if (tid == 0 && alive) {
      if (!first) product(tmem, b1, b2);       // P Q
      if (!last) product(tmem + 128, b0, b1);   // A P
      go(0);
    }
    ok = wait(0);
    if (ok && in_rows) {
      const float fq = f.chain, fw = f.inner;
      for (int c = quarter * 32; c < min(mk, quarter * 32 + 32); c += 16) {
        float y[16];
        if (!first) {
          __syncwarp();
          tmem_load16(tmem_row + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) y[q] *= fq;
          store_pair(b2, row, c / 8, y);
          store_pair(b2, row, c / 8 + 1, y + 8);
        }
        if (!last) {
          __syncwarp();
          tmem_load16(tmem_row + 128 + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) y[q] *= fw;
          store_pair(b0, row, c / 8, y);
          store_pair(b0, row, c / 8 + 1, y + 8);
        }
      }
    }
    ready(ok);
    if (last) break;
    if (tid == 0 && alive) {
      product(tmem, b1, b0);  // P (A P)
      go(0);
    }
    ok = wait(0);
    if (ok && in_rows) {
      for (int c = quarter * 32; c < min(mk, quarter * 32 + 32); c += 16) {
        float y[16];
        __syncwarp();
        tmem_load16(tmem_row + c, y);
#pragma unroll
        for (int q = 0; q < 16; ++q) y[q] *= f.next;
        store_pair(b0, row, c / 8, y);
        store_pair(b0, row, c / 8 + 1, y + 8);
      }
    }
    ready(ok);
  }

  // ---- Q X, slice after slice, the epilogue one slice behind the products -------
  const float to_result = a.step_factors[end - 1].result;
  used = 0;
  for (int j0 = rank * kSlice;; j0 += kCtas * kSlice, ++used) {
    const int i = used & 1;
    const bool more = j0 < x.n;
    if (!more && used == 0) break;
    if (more) {
      fetch(j0, i ? b1 : b0);
      ready(alive);
      if (tid == 0 && alive) {
        issue_pair(tmem + i * 128, b2, i ? b1 : b0, false, kSlice, mk, false);
        mma_commit<1>(smem_u32(&sh.bar[1 + i]));
      }
    }
    if (used > 0) {
      const int before = j0 - kCtas * kSlice;
      ok = wait(2 - i);
      if (ok && in_rows) {
#pragma unroll 1
        for (int c = quarter * 32; c < quarter * 32 + 32; c += 16) {
          float y[16];
          __syncwarp();
          tmem_load16(tmem_row + (1 - i) * 128 + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) y[q] *= to_result;
          if (end == a.steps) {
            store_result<kMuon>(a, mat, x, vec, row, before + c, y);
            store_result<kMuon>(a, mat, x, vec, row, before + c + 8, y + 8);
          } else {
            store_iterate(xw, work, row, before + c, y);
            store_iterate(xw, work, row, before + c + 8, y + 8);
          }
        }
      }
      ready(ok);
    }
    if (!more) break;
  }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 0) tmem_free<1>(tmem, kTmemColumns);
  // no CTA leaves while another may read its shared memory (the last such read
  // lies before the barrier behind the joined Gram matrix)
}

template <int kCtas, bool kMuon, bool kFp32>
cudaError_t launch(const ThinArgs& a, long long mats, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(ns_thin_kernel<kCtas, kMuon, kFp32>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(mats * kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ns_thin_kernel<kCtas, kMuon, kFp32>, a);
}

template <bool kMuon, bool kFp32>
cudaError_t launch_ctas(const ThinArgs& a, int ctas, long long mats, cudaStream_t stream) {
  switch (ctas) {
    case 1: return launch<1, kMuon, kFp32>(a, mats, stream);
    case 2: return launch<2, kMuon, kFp32>(a, mats, stream);
    case 4: return launch<4, kMuon, kFp32>(a, mats, stream);
    default: return launch<8, kMuon, kFp32>(a, mats, stream);
  }
}

}  // namespace

// By the shape alone (not by how many matrices there are), so that a matrix
// gives the same bits in any company.
int thin_ctas(long long rows, long long cols) {
  const long long slices = ((rows > cols ? rows : cols) + kSlice - 1) / kSlice;
  return slices <= 1 ? 1 : slices <= 2 ? 2 : slices <= 4 ? 4 : 8;
}

cudaError_t launch_ns_thin(const ThinArgs& a, bool muon, int ctas, long long mats, cudaStream_t stream, int* launches) {
  ++*launches;
  if (muon) return launch_ctas<true, true>(a, ctas, mats, stream);
  return a.src.fp32 ? launch_ctas<false, true>(a, ctas, mats, stream) : launch_ctas<false, false>(a, ctas, mats, stream);
}

unsigned int thin_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

unsigned int thin_debug_failures() {
#ifdef ZFS_DEBUG_CHECKS
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_debug_failures, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
#else
  return 0;
#endif
}

}  // namespace zfs
