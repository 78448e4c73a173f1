// Newton-Schulz orthogonalisation of thin matrices, smaller side m <= kThin:
// the whole chain in one launch, a cluster of CTAs per matrix.
//
//   A = X X^T,  P = a I + b A + c A A,  X <- P X      (steps times)
//
// What bounds it is latency: a product of 128 takes under half a microsecond,
// and the next one waits for it.  Hence one launch; A, P and X stay in shared
// memory, the columns of X split over up to 8 CTAs in slices of 128 whose
// partial Gram matrices are joined in distributed shared memory; every CTA
// forms P by itself rather than wait for another.  More than one slice per CTA
// (n > 1024) pass through global memory as ready images, once per step: a
// slice's new columns go straight into the next step's Gram matrix.  In the
// Muon step the momentum pass is the first thing the kernel does.  Five steps on
// one 64 x 64 matrix take 21 us with the call, and a whole step of an MLP of
// five layers up to 128 wide 43 us; with a launch per product one 128 x 512
// matrix would be 17 of them at some 7 us.
//
// With tiny m the roundings of a step do not average out, and latency leaves
// room, so products keep 22 bits here: every operand is an fp16 pair (hi + lo)
// and a product is hi lo + lo hi + hi hi with fp32 sums (which the tensor cores
// truncate: 1e-6): 1e-5 off after five steps where 11 bits leave 5e-3.

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
  float sum;  // of this CTA's columns, read by the cluster
  float warp_sum[kWarps];
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

// acc (128 rows, `n` columns, a multiple of 16) = sum over k < 64 kBlocks of the
// pair product of two buffers, A K-major and B K-major or MN-major.  One
// thread, straight-line code with descriptors that move by constants: what this
// thread does between two MMAs is what a short product takes (predicated
// pieces of 16 took 1550 cycles whatever the depth).
template <int kBlocks>
__device__ __forceinline__ void issue_blocks(uint32_t acc, uint64_t da, uint64_t db, uint32_t b_step, uint32_t b_block,
                                             uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int part = 0; part < 3; ++part) {  // hi lo, lo hi, hi hi: the small terms first, as sums are truncated
    const uint64_t pa = da + (part == 1 ? kHalfBytes >> 4 : 0), pb = db + (part == 0 ? kHalfBytes >> 4 : 0);
#pragma unroll
    for (int block = 0; block < kBlocks; ++block) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t ka = pa + block * (kBlockBytes >> 4) + 2 * k, kb = pb + block * b_block + k * b_step;
        if (part == 0 && block == 0 && k == 0) mma<1>(acc, ka, kb, idesc, accumulate);
        else mma_add<1>(acc, ka, kb, idesc);
      }
    }
  }
}
// `deep`: more than 64 of k; what the operands hold beyond their size is zero.
__device__ __forceinline__ void issue_pair(uint32_t acc, uint32_t a, uint32_t b, bool b_k_major, int n, bool deep,
                                           bool accumulate) {
  const uint32_t idesc = (1u << 4) | (b_k_major ? 0u : 1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
  const uint64_t da = smem_desc(a, true, 0), db = smem_desc(b, b_k_major, kBlockBytes);
  const uint32_t b_step = b_k_major ? 2 : 128, b_block = b_k_major ? kBlockBytes >> 4 : 512;  // units of 16 bytes
  if (deep) issue_blocks<2>(acc, da, db, b_step, b_block, idesc, accumulate);
  else issue_blocks<1>(acc, da, db, b_step, b_block, idesc, accumulate);
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

// A run of the slice from column j0, scaled (by a power of two first), as pairs
// in `buffer`.
__device__ __forceinline__ void put_run(const Matrix& x, const Run& r, int j0, float power, float scale, float* v,
                                        uint32_t buffer) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = v[k] * power * scale;
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

// A thread's sum of squares, entry after entry.  Every 32 slices `part` moves to
// `sum`, with what the additions round off kept beside it: many slices are long runs.
struct LongSum {
  float part = 0.0f, sum = 0.0f, rounded = 0.0f;
  __device__ __forceinline__ void end_slice(int s) {
    if (s % 32 != 31) return;
    const float to = __fadd_rn(sum, part), added = __fsub_rn(to, sum);
    rounded += __fadd_rn(__fsub_rn(sum, __fsub_rn(to, added)), __fsub_rn(part, added));
    sum = to;
    part = 0.0f;
  }
  __device__ __forceinline__ float value() const { return part + rounded + sum; }
};

// A thread's sum over its CTA's slices once more, of entries times `power` (not
// inline: for matrices that hardly ever come).
template <bool kFp32>
__device__ __noinline__ float scaled_squares(const void* base, const Matrix x, bool vec, int j0, int step, int slices,
                                             float power) {
  LongSum sum;
  const int runs = slice_runs(x);
  for (int s = 0; s < slices; ++s) {
    for (int i = threadIdx.x; i < runs; i += kThreads) {
      float v[8];
      load_run<kFp32>(base, slice_run(x, j0 + s * step, i), vec, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum.part += v[k] * power * (v[k] * power);
    }
    sum.end_slice(s);
  }
  return sum.value();
}

// The momentum pass of a run: y becomes the update (the squares' sum is the caller's).
template <bool kFp32>
__device__ __forceinline__ void momentum_run(const ThinArgs& a, int mat, const Run& r, bool vec, float clip, float* y,
                                             unsigned* nf) {
  const long long base = a.offset[mat];
  float g[8], m[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = 0.0f;
  if (r.count == 0 || !ZFS_CHECK(base >= 0 && base + r.at + r.count <= a.total_padded)) return;
  load_run<true>(a.mom + base, r, vec, m);
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
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (a.clip) g[k] = __fmul_rn(g[k], clip);
    m[k] = __fadd_rn(__fmul_rn(a.mu, m[k]), g[k]);
    y[k] = a.nesterov ? __fadd_rn(g[k], __fmul_rn(a.mu, m[k])) : m[k];
  }
  float* mom = a.mom + base + r.at;
  if (vec && r.count == 8) {
    reinterpret_cast<float4*>(mom)[0] = make_float4(m[0], m[1], m[2], m[3]);
    reinterpret_cast<float4*>(mom)[1] = make_float4(m[4], m[5], m[6], m[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < r.count) mom[k] = m[k];
  }
}

// ---- the output --------------------------------------------------------------
// One finished value at `at` of the matrix's storage.
template <bool kMuon>
__device__ __forceinline__ void put_value(const ThinArgs& a, int mat, long long at, float y, float old) {
  if constexpr (kMuon) {
    const float z = __fadd_rn(__fmul_rn(old, a.decay), __fmul_rn(-a.step[mat], y));
    a.master[a.offset[mat] + at] = z;
    a.p16[a.offset[mat] + at] = to_bf16_bits(z);
  } else {
    a.out[mat * a.out_mat_stride + at] = to_bf16_bits(y);
  }
}
template <bool kMuon>
__device__ __forceinline__ float old_value(const ThinArgs& a, int mat, long long at, bool* ok) {
  if constexpr (kMuon) {
    *ok = ZFS_CHECK(a.offset[mat] + at >= 0 && a.offset[mat] + at < a.total_padded);
    return *ok ? a.master[a.offset[mat] + at] : 0.0f;
  } else {
    *ok = true;
    return 0.0f;
  }
}

// A slice of a wide matrix from `rows` (fp32, 128 x 128, 16-byte pieces
// swizzled by row): a row per warp, so that accesses are contiguous.
template <bool kMuon>
__device__ __forceinline__ void write_rows(const ThinArgs& a, int mat, const Matrix& x, bool vec, uint32_t rows, int j0,
                                           int warp, int lane) {
  const long long ld = kMuon ? x.ld : a.out_row_stride;
  const int width = min(kSlice, x.n - j0);
  if ((kMuon ? vec : a.vec_out != 0) && width == kSlice) {
#pragma unroll 2
    for (int i = warp; i < x.m; i += kWarps) {
      const long long at = i * ld + j0 + 4 * lane;
      const uint4 v = lds16(rows + i * 512 + ((lane ^ (i & 7)) << 4));
      float4 y = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
      if constexpr (kMuon) {
        const long long to = a.offset[mat] + at;
        if (!ZFS_CHECK(to >= 0 && to + 4 <= a.total_padded)) continue;
        const float4 old = *reinterpret_cast<const float4*>(a.master + to);
        const float step = -a.step[mat];
        y.x = __fadd_rn(__fmul_rn(old.x, a.decay), __fmul_rn(step, y.x));
        y.y = __fadd_rn(__fmul_rn(old.y, a.decay), __fmul_rn(step, y.y));
        y.z = __fadd_rn(__fmul_rn(old.z, a.decay), __fmul_rn(step, y.z));
        y.w = __fadd_rn(__fmul_rn(old.w, a.decay), __fmul_rn(step, y.w));
        *reinterpret_cast<float4*>(a.master + to) = y;
        *reinterpret_cast<uint2*>(a.p16 + to) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      } else {
        *reinterpret_cast<uint2*>(a.out + mat * a.out_mat_stride + at) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      }
    }
  } else {
    for (int i = warp; i < x.m; i += kWarps) {
#pragma unroll
      for (int q = 0; q < kSlice / 32; ++q) {
        const int c = lane + 32 * q;
        if (c >= width) continue;
        float y;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(y)
                     : "r"(rows + i * 512 + (((c / 4) ^ (i & 7)) << 4) + c % 4 * 4)
                     : "memory");
        bool ok;
        const float old = old_value<kMuon>(a, mat, i * ld + j0 + c, &ok);
        if (ok) put_value<kMuon>(a, mat, i * ld + j0 + c, y, old);
      }
    }
  }
}

// Sixteen columns from j of X row i of a tall matrix: lanes are consecutive
// elements of its rows.
template <bool kMuon>
__device__ __forceinline__ void write_columns(const ThinArgs& a, int mat, const Matrix& x, int i, int j, const float* y) {
  if (i >= x.m) return;
  const long long ld = kMuon ? x.ld : a.out_row_stride;
  float old[16];
  bool ok[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    ok[k] = false;
    if (j + k < x.n) old[k] = old_value<kMuon>(a, mat, (j + k) * ld + i, &ok[k]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (ok[k]) put_value<kMuon>(a, mat, (j + k) * ld + i, y[k], old[k]);
}

// ---- the kernel --------------------------------------------------------------
// kCtas CTAs per matrix.  Every CTA of a cluster reaches every cluster barrier;
// one whose wait gave up (alive = false) only skips its work.
template <int kCtas, bool kMuon, bool kFp32>
__global__ void __launch_bounds__(kThreads, 1) ns_thin_kernel(const __grid_constant__ ThinArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sh;
  if constexpr (kMuon) {
    asm volatile("griddepcontrol.launch_dependents;");
    if (a.dev_t && *a.dev_t >= a.dev_steps) {  // the same for the whole grid
      asm volatile("griddepcontrol.wait;" ::: "memory");
      return;
    }
  }
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = kCtas > 1 ? cluster_rank() : 0;
  const int mat = blockIdx.x / kCtas;
  // A, then P, in square; slices of X in turn in the other two
  const uint32_t square = (smem_u32(smem_raw) + 1023) & ~1023u, slices = square + kPairBytes;
  Matrix x;
  {
    const int at = kMuon ? mat : 0, rows = a.rows[at], cols = a.cols[at];
    x.tall = rows > cols;
    x.m = min(rows, cols);
    x.n = max(rows, cols);
    x.mk = (x.m + 15) / 16 * 16;
    x.ld = kMuon ? cols : a.src.row_stride;
  }
  const int mk = x.mk, all = (x.n + kSlice - 1) / kSlice;
  const int mine = (all - static_cast<int>(rank) + kCtas - 1) / kCtas;  // slices rank, rank + kCtas, ...
  const bool many = all > kCtas;  // some CTA has more than one: the images pass through global memory
  const bool vec = kMuon ? (a.vec[mat / 32] >> (mat % 32)) & 1 : a.src.vec_ok != 0;
  // of this matrix: the Muon step's update (fp32, only with many slices), then the images
  char* work = a.work + (kMuon ? a.work_offset[mat] : mat * a.work_mat_stride);
  float* update = reinterpret_cast<float*>(work);
  char* images = work + (kMuon ? (static_cast<long long>(x.m) * x.n * 4 + 255) / 256 * 256 : 0);
  const void* source = kMuon ? static_cast<const void*>(update)
                             : static_cast<const char*>(a.src.data) + mat * a.src.mat_stride * (kFp32 ? 4 : 2);
  if (tid == 0) {
    sh.gave_up = 0;
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&sh.bar[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc<1>(smem_u32(&sh.tmem), kTmemColumns);
  // Products run over 64 or 128 of k: what lies beyond mk (columns of A and P,
  // rows of X) is zero.  Later writes stay within mk; a slice buffer that took
  // other data is cleared again (clear_rest).
  if (mk % 64 != 0) {
    for (uint32_t i = tid; i < 3 * kPairBytes / 16; i += kThreads) sts16(square + 16 * i, make_uint4(0, 0, 0, 0));
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sh.tmem, gram = tmem, other = tmem + 128;
  bool alive = true;
  // Barriers: products that a buffer of slices (0, 1) waits for, all others (2).
  uint32_t phase[3] = {0, 0, 0};
  bool pending[2] = {false, false};
  auto wait = [&](int i) {  // all threads
    const bool ok = alive && wait_phase(smem_u32(&sh.bar[i]), phase[i], &sh.gave_up);
    phase[i] ^= 1;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    return ok;
  };
  auto drained = [&](int i) {  // the Gram products of slice buffer i
    const bool ok = !pending[i] || wait(i);
    pending[i] = false;
    return ok;
  };
  // Makes shared-memory operands and drained accumulators ready for products.
  auto ready = [&](bool ok) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    alive = __syncthreads_and(ok ? 1 : 0) != 0;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  };
  auto first_column = [&](int s) { return (static_cast<int>(rank) + s * kCtas) * kSlice; };
  auto depth_of = [&](int s) { return (min(kSlice, x.n - first_column(s)) + 15) / 16 * 16; };
  auto image = [&](int s) { return images + (static_cast<long long>(rank) + s * kCtas) * (512LL * mk); };
  // A slice's image between shared and global memory: mk rows of the four blocks.
  auto store_image = [&](int s, uint32_t from) {  // one thread
    for (int b = 0; b < 4; ++b)
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(image(s) + b * 128LL * mk),
                   "r"(from + b * kBlockBytes), "r"(128 * mk)
                   : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  };
  auto load_image = [&](int s, uint32_t to) {  // one thread
    const uint32_t bar = smem_u32(&sh.bar[2]);
    mbar_expect_tx(bar, 512 * mk);
    for (int b = 0; b < 4; ++b)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       to + b * kBlockBytes),
                   "l"(image(s) + b * 128LL * mk), "r"(128 * mk), "r"(bar)
                   : "memory");
  };
  // Zero from row mk on in the blocks of a slice buffer, as far as products read.
  auto clear_rest = [&](uint32_t buffer) {
    const int top = mk > 64 ? 128 : 64, pieces = (top - mk) * 8;
    for (int e = tid; e < 4 * pieces; e += kThreads)
      sts16(buffer + e / pieces * kBlockBytes + mk * 128 + e % pieces * 16, make_uint4(0, 0, 0, 0));
  };
  // the share of a thread in an epilogue: row `row`, columns from `begin`
  const int row = (warp % 4) * 32 + lane, quarter = warp / 4;
  const bool in_rows = (warp % 4) * 32 < mk;  // the same for the whole warp
  const uint32_t lanes = ((warp % 4) * 32) << 16;
  const int share = (mk / 16 + 3) / 4 * 16;   // columns of a quarter of an m x m matrix
  auto add_to_gram = [&](int s, uint32_t buffer) {  // one thread
    issue_pair(gram, buffer, buffer, true, mk, depth_of(s) > 64, s > 0);
    mma_commit<1>(smem_u32(&sh.bar[s & 1]));
  };

  // ---- norm (and momentum) ------------------------------------------------------
  // A single slice stays in registers until the norm is known.
  const float clip = kMuon && a.clip ? *a.clip : 1.0f;
  const int runs = slice_runs(x);
  constexpr int kHeld = kThin * (kSlice / 8) / kThreads;
  float held[kHeld][8];
  unsigned nf = 0;
  LongSum sum;
  // The sum over the cluster, in one order for every thread of it.
  auto joined = [&](float value) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) value += __shfl_xor_sync(0xffffffffu, value, o);
    if (lane == 0) sh.warp_sum[warp] = value;
    __syncthreads();
    value = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) value += sh.warp_sum[w];
    if constexpr (kCtas > 1) {
      if (tid == 0) sh.sum = value;
      cluster_sync();
      value = 0.0f;
      for (int r = 0; r < kCtas; ++r) value += ld_cluster(map_rank(smem_u32(&sh.sum), r));
    }
    return value;
  };
  for (int s = 0; s < mine; ++s) {
    const int j0 = first_column(s);
#pragma unroll
    for (int q = 0; q < kHeld; ++q) {
      const int i = tid + q * kThreads;
      if (i < runs) {
        const Run r = slice_run(x, j0, i);
        if constexpr (kMuon) {
          if (a.grad_fp32) momentum_run<true>(a, mat, r, vec, clip, held[q], &nf);
          else momentum_run<false>(a, mat, r, vec, clip, held[q], &nf);
          if (many) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < r.count) update[r.at + k] = held[q][k];
          }
        } else {
          load_run<kFp32>(source, r, vec, held[q]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum.part += held[q][k] * held[q][k];
      }
    }
    sum.end_slice(s);
  }
  if constexpr (kMuon) flush_nonfinite(a.nonfinite, nf);
  float power = 1.0f, total = joined(sum.value());
  // The same for the whole cluster; as a vote, so that the compiler knows it to be
  // the same for a warp (the barriers in the branch cost every call 1.5 us else).
  if (__any_sync(0xffffffffu, !(total >= kNormLow && total <= kNormHigh))) {
    power = total < kNormLow ? kNormUp : kNormDown;
    float again = 0.0f;
    if (many) {
      again = scaled_squares<kMuon || kFp32>(kMuon ? update : source, x, vec, first_column(0), kCtas * kSlice, mine, power);
    } else if (mine > 0) {
#pragma unroll
      for (int q = 0; q < kHeld; ++q) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (tid + q * kThreads < runs) again += held[q][k] * power * (held[q][k] * power);
      }
    }
    if constexpr (kCtas > 1) cluster_sync();  // the first sums have been read
    else __syncthreads();
    total = joined(again);
  }
  // x / (norm + eps), both times `power`
  const float norm = sqrtf(total) + a.eps * power;
  const float scale = norm == 0.0f ? 0.0f : 1.0f / norm * a.step_factors[0].x;  // a zero matrix stays one

  // ---- X0 and its Gram matrix ---------------------------------------------------
  bool ok = alive;
  for (int s = 0; s < mine; ++s) {
    const int j0 = first_column(s), i = s & 1;
    const uint32_t buffer = slices + i * kPairBytes;
    if (many) {
      ok = drained(i);
      if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kHeld; ++q) {
      const int e = tid + q * kThreads;
      if (e < runs) {
        const Run r = slice_run(x, j0, e);
        if (many) {
          if constexpr (kMuon) load_run<true>(update, r, false, held[q]);
          else load_run<kFp32>(source, r, vec, held[q]);
        }
        put_run(x, r, j0, power, scale, held[q], buffer);
      }
    }
    ready(ok);
    if (tid == 0 && alive) {
      if (many) store_image(s, buffer);
      add_to_gram(s, buffer);
    }
    pending[i] = true;
  }

  for (int k = 0; k < a.steps; ++k) {
    const ThinStep& f = a.step_factors[k];
    const bool last = k + 1 == a.steps;
    ok = drained(0);
    ok = drained(1) && ok;
    if (many && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");

    // ---- A, joined over the cluster -----------------------------------------------
    if constexpr (kCtas == 1) {
      if (ok && in_rows) {
        for (int c = quarter * share; c < min(mk, (quarter + 1) * share); c += 16) {
          float y[16];
          __syncwarp();
          tmem_load16(gram + lanes + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) y[q] *= f.gram;
          store_pair(square, row, c / 8, y);
          store_pair(square, row, c / 8 + 1, y + 8);
        }
      }
    } else {
      // Partial sums to this CTA's second slice buffer (column after column: A
      // is symmetric, and lanes are rows); each CTA joins mk / kCtas columns
      // in rank order and gives them to all.
      const uint32_t partial = slices + kPairBytes;
      __syncthreads();  // (with many slices: the last image has been stored)
      if (ok && in_rows) {
        for (int c = quarter * share; c < min(mk, (quarter + 1) * share); c += 16) {
          float y[16];
          __syncwarp();
          tmem_load16(gram + lanes + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(partial + ((c + q) * 128 + row) * 4),
                         "f"(mine > 0 ? y[q] * f.gram : 0.0f)
                         : "memory");
        }
      }
      cluster_sync();
      const int columns = mk / kCtas, from = rank * columns;
      for (int e = tid; e < columns * (mk / 2); e += kThreads) {
        const int c = from + e / (mk / 2), r = e % (mk / 2) * 2;
        float u = 0.0f, v = 0.0f;
#pragma unroll
        for (int q = 0; q < kCtas; ++q) {
          const uint32_t at = map_rank(partial + (c * 128 + r) * 4, q);
          u += ld_cluster(at);
          v += ld_cluster(at + 4);
        }
        const uint32_t hi = half2_bits(u, v);
        const float2 h = half2_values(hi);
        const uint32_t lo = half2_bits(u - h.x, v - h.y);
        const uint32_t at = chunk_at(square, c, r / 8) + r % 8 * 2;  // row c of A, columns r and r + 1
#pragma unroll
        for (int q = 0; q < kCtas; ++q) {
          st_cluster(map_rank(at, q), hi);
          st_cluster(map_rank(at + kHalfBytes, q), lo);
        }
      }
      asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
      cluster_sync();
      if (many) clear_rest(partial);
    }
    ready(ok);

    // ---- P over A -----------------------------------------------------------------
    if (tid == 0 && alive) {
      issue_pair(other, square, square, true, mk, mk > 64, false);
      mma_commit<1>(smem_u32(&sh.bar[2]));
    }
    ok = wait(2);
    if (ok && in_rows) {
      for (int c = quarter * share; c < min(mk, (quarter + 1) * share); c += 16) {
        float y[16];
        __syncwarp();
        tmem_load16(other + lanes + c, y);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float old[8];
          load_pair(square, row, c / 8 + h, old);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int col = c + 8 * h + q;
            y[8 * h + q] = fmaf(f.square, y[8 * h + q], f.gram_term * old[q]) +
                           (col == row && row < x.m ? f.identity : 0.0f);
          }
          store_pair(square, row, c / 8 + h, y + 8 * h);
        }
      }
    }
    ready(ok);

    // ---- P X, slice after slice ------------------------------------------------------
    for (int s = 0; s < mine; ++s) {
      const int j0 = first_column(s), i = s & 1, width = depth_of(s);
      const uint32_t buffer = slices + i * kPairBytes, beside = slices + (1 - i) * kPairBytes;
      if (many) {
        ok = drained(i);
        if (tid == 0) {
          // the buffer's image has been stored; a load's bytes count on barrier 2
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          if (ok && alive) load_image(s, buffer);
        }
        ok = wait(2) && ok;
        ready(ok);
      }
      if (tid == 0 && alive) {
        issue_pair(other, square, buffer, false, width, mk > 64, false);
        mma_commit<1>(smem_u32(&sh.bar[2]));
      }
      ok = wait(2);
      if (last && !x.tall && many) {  // the buffer beside takes the finished rows
        ok = drained(1 - i) && ok;
        __syncthreads();
      }
      if (ok && in_rows) {
        for (int c = quarter * 32; c < min(width, quarter * 32 + 32); c += 16) {
          float y[16];
          __syncwarp();
          tmem_load16(other + lanes + c, y);
#pragma unroll
          for (int q = 0; q < 16; ++q) y[q] *= f.result;
          if (!last) {
            store_pair(buffer, row, c / 8, y);
            store_pair(buffer, row, c / 8 + 1, y + 8);
          } else if (x.tall) {
            write_columns<kMuon>(a, mat, x, row, j0 + c, y);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sts16(beside + row * 512 + (((c / 4 + q) ^ (row & 7)) << 4),
                    make_uint4(__float_as_uint(y[4 * q]), __float_as_uint(y[4 * q + 1]), __float_as_uint(y[4 * q + 2]),
                               __float_as_uint(y[4 * q + 3])));
          }
        }
      }
      ready(ok);
      if (!last) {
        if (tid == 0 && alive) {
          if (many) store_image(s, buffer);
          add_to_gram(s, buffer);
        }
        pending[i] = true;
      } else if (!x.tall) {
        if (alive) write_rows<kMuon>(a, mat, x, vec, beside, j0, warp, lane);
        if (many) {
          __syncthreads();
          clear_rest(beside);
          ready(alive);
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 0) tmem_free<1>(tmem, kTmemColumns);
  if (many && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  // No CTA leaves while another may read its shared memory: the last such read
  // lies before the barrier behind the last joined Gram matrix.
  // Launched beside a kernel of the same step: what waits for this one may rely
  // on that one too.
  if constexpr (kMuon) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int kCtas, bool kMuon, bool kFp32>
cudaError_t launch(const ThinArgs& a, long long mats, bool follows, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(ns_thin_kernel<kCtas, kMuon, kFp32>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(mats * kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = follows ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ns_thin_kernel<kCtas, kMuon, kFp32>, a);
}

template <bool kMuon, bool kFp32>
cudaError_t launch_ctas(const ThinArgs& a, int ctas, long long mats, bool follows, cudaStream_t stream) {
  switch (ctas) {
    case 1: return launch<1, kMuon, kFp32>(a, mats, follows, stream);
    case 2: return launch<2, kMuon, kFp32>(a, mats, follows, stream);
    case 4: return launch<4, kMuon, kFp32>(a, mats, follows, stream);
    default: return launch<8, kMuon, kFp32>(a, mats, follows, stream);
  }
}

}  // namespace

// By the shape alone (not by how many matrices there are), so that a matrix
// gives the same bits in any company.
int thin_ctas(long long rows, long long cols) {
  const long long slices = ((rows > cols ? rows : cols) + kSlice - 1) / kSlice;
  return slices <= 1 ? 1 : slices <= 2 ? 2 : slices <= 4 ? 4 : 8;
}

// What a matrix needs of the workspace: nothing while every CTA has one slice;
// else the images of the slices and, in a Muon step, the update.
long long thin_work(long long rows, long long cols, bool muon) {
  const long long m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  const long long all = (n + kSlice - 1) / kSlice, mk = (m + 15) / 16 * 16;
  if (all <= thin_ctas(rows, cols)) return 0;
  return all * 512 * mk + (muon ? (m * n * 4 + 255) / 256 * 256 : 0);
}

cudaError_t launch_ns_thin(const ThinArgs& a, bool muon, bool follows, int ctas, long long mats, cudaStream_t stream,
                           int* launches) {
  ++*launches;
  if (muon) return launch_ctas<true, true>(a, ctas, mats, follows, stream);
  return a.src.fp32 ? launch_ctas<false, true>(a, ctas, mats, false, stream)
                    : launch_ctas<false, false>(a, ctas, mats, false, stream);
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
