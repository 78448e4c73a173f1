// Elementwise passes around the Newton-Schulz orthogonalisation: the Muon
// momentum pass over the flat buffer, the Frobenius norm of a stack of
// matrices, and its normalisation into scaled fp16 pairs.
//
// All are one pass over memory-resident data and bound by it; the norm is
// summed per chunk of kNsChunk elements of a matrix, in fp32 over the elements
// of a warp and in fp64 above, each in a fixed order, whatever the entries' size.
// A CTA per chunk keeps two vectors of every replica in flight per thread.  Over
// 486 M elements of 8 bf16 replicas the momentum pass (28 bytes per element) takes
// 1.96 ms, 6.9 TB/s, and the normalisation (8 bytes) 0.61 ms, 6.4 TB/s; 71 M
// elements in four launches each, one after another, 348 us (5.7 TB/s) and 104 us
// (5.5); they overlap in a step (zero_runtime.cpp), which takes 40 us less for it.
// Matrices that are not 16-byte aligned go element by element (the whole step of the
// 71 M elements 2.6 ms instead of 1.75).

#include <cuda_fp16.h>

#include "zero_device.cuh"
#include "zero_muon_internal.h"

namespace zfs {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = static_cast<int>(kNsChunk) / kThreads;  // elements per thread and chunk
static_assert(kPerThread % kVec == 0, "whole vectors per thread");

// A thread's sum of squares, entry after entry.  Vectors that leave it outside
// kNormLow..kNormHigh are summed apart, from their entries times a power of two, and
// one such sum is enough: beside large ones (odd < 0: minus the sum of
// (x kNormDown)^2) small ones (odd > 0: (x kNormUp)^2) are nothing.
struct Squares {
  float sum = 0.0f, odd = 0.0f;  // sum: 0 or in the range
  __device__ __forceinline__ void add(const float* x) {
    float s = sum;
#pragma unroll
    for (int k = 0; k < kVec; ++k) s += x[k] * x[k];
    if (s >= kNormLow && s <= kNormHigh) {
      sum = s;
      return;
    }
    const bool small = s < kNormLow;
    const float f = small ? kNormUp : kNormDown;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kVec; ++k) s += x[k] * f * (x[k] * f);
    if (!small) odd = (odd > 0.0f ? 0.0f : odd) - s;
    else if (odd >= 0.0f) odd += s;
  }
};

// The CTA's sum of squares in a fixed order, fp32 within a warp and fp64 above
// (by one thread: the GPU has few fp64 units); valid in thread 0.
__device__ __forceinline__ double block_sum(const Squares& q) {
  __shared__ float warp_sum[kThreads / 32];
  float x = q.sum;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_down_sync(0xffffffffu, x, o);
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = x;
  const bool odd = __syncthreads_or(q.odd != 0.0f) != 0;
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += warp_sum[w];
  }
  if (__builtin_expect(odd, 0)) {
    __shared__ double odd_sum[kThreads / 32];
    constexpr double kUp = static_cast<double>(kNormUp) * kNormUp, kDown = static_cast<double>(kNormDown) * kNormDown;
    double y = q.odd >= 0.0f ? q.odd / kUp : -q.odd / kDown;
    for (int o = 16; o > 0; o >>= 1) y += __shfl_down_sync(0xffffffffu, y, o);
    if (threadIdx.x % 32 == 0) odd_sum[threadIdx.x / 32] = y;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < kThreads / 32; ++w) s += odd_sum[w];
    }
  }
  return s;
}

// One chunk of one matrix per CTA (grid: chunk, matrix).  A thread's vectors
// are kThreads vectors apart, so a warp reads contiguous runs.  The CTAs per SM are
// what keeps the loads in flight (bf16 vectors at five instead of six: 5 % slower).
template <bool kFp32, bool kVecOk>
__global__ void __launch_bounds__(kThreads, kVecOk && !kFp32 ? 6 : 5) momentum_kernel(const __grid_constant__ MomentumArgs a) {
  if (a.dev_t && *a.dev_t >= a.dev_steps) {  // capturable: past the captured steps' table
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int mat = blockIdx.y;
  const float clip = a.clip ? *a.clip : 1.0f;
  const long long base = a.offset[mat];
  unsigned nf = 0;
  Squares sq;
#pragma unroll 2
  for (int i = 0; i < kPerThread / kVec; ++i) {
    const long long e = blockIdx.x * kNsChunk + (static_cast<long long>(i) * kThreads + threadIdx.x) * kVec;
    if (e >= a.numel) continue;
    const int count = static_cast<int>(a.numel - e < kVec ? a.numel - e : kVec);
    if (!ZFS_CHECK(base >= 0 && base + e + count <= a.total_padded)) continue;
    float g[kVec], x[kVec], m[kVec];
    load8<kFp32, kVecOk>(a.g[mat][0], e, count, g);
    for (int r = 1; r < a.n_ranks; ++r) {
      load8<kFp32, kVecOk>(a.g[mat][r], e, count, x);
#pragma unroll
      for (int k = 0; k < kVec; ++k) g[k] = __fadd_rn(g[k], x[k]);
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) g[k] = __fmul_rn(g[k], a.inv_n);
    nf += tally_nonfinite<kVec>(g);
    load8<true, kVecOk>(a.mom, base + e, count, m);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      if (a.clip) g[k] = __fmul_rn(g[k], clip);
      m[k] = __fadd_rn(__fmul_rn(a.mu, m[k]), g[k]);
      x[k] = a.nesterov ? __fadd_rn(g[k], __fmul_rn(a.mu, m[k])) : m[k];
    }
    sq.add(x);
    float* mom = a.mom + base + e;
    float* upd = a.update + mat * a.numel + e;
    if constexpr (kVecOk) {
      reinterpret_cast<float4*>(mom)[0] = make_float4(m[0], m[1], m[2], m[3]);
      reinterpret_cast<float4*>(mom)[1] = make_float4(m[4], m[5], m[6], m[7]);
      reinterpret_cast<float4*>(upd)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(upd)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        if (k < count) {
          mom[k] = m[k];
          upd[k] = x[k];
        }
      }
    }
  }
  flush_nonfinite(a.nonfinite, nf);
  const double s = block_sum(sq);
  if (threadIdx.x == 0) a.partials[mat * a.chunks + blockIdx.x] = s;
  // Launched beside the normalisation of another stack: what waits for this
  // kernel may rely on that one too.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Eight consecutive elements of the stack in logical (row-major) order.
template <bool kFp32, bool kVecOk>
__device__ __forceinline__ void load_logical(const MatSource& s, int mat, long long cols, long long e, int count,
                                             float* x) {
  const long long row = e / cols, col = e - row * cols;
  if (col + count <= cols) {
    load8<kFp32, kVecOk>(s.data, mat * s.mat_stride + row * s.row_stride + col, count, x);
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      x[k] = 0.0f;
      if (k < count) {
        const long long r = (e + k) / cols, c = (e + k) - r * cols;
        float one[8];
        load8<kFp32, false>(s.data, mat * s.mat_stride + r * s.row_stride + c, 1, one);
        x[k] = one[0];
      }
    }
  }
}

template <bool kFp32, bool kVecOk>
__global__ void __launch_bounds__(kThreads, 8)
    ns_norm_kernel(const MatSource s, long long cols, long long numel, long long chunks, double* partials) {
  const int mat = blockIdx.y;
  Squares sq;
#pragma unroll 2
  for (int i = 0; i < kPerThread / kVec; ++i) {
    const long long e = blockIdx.x * kNsChunk + (static_cast<long long>(i) * kThreads + threadIdx.x) * kVec;
    if (e >= numel) continue;
    const int count = static_cast<int>(numel - e < kVec ? numel - e : kVec);
    float x[kVec];
    load_logical<kFp32, kVecOk>(s, mat, cols, e, count, x);
    sq.add(x);
  }
  const double sum = block_sum(sq);
  if (threadIdx.x == 0) partials[mat * chunks + blockIdx.x] = sum;
}

// X0 = source / (norm + eps), stored as hi + lo: hi the nearest fp16 of the
// scaled value, lo the nearest fp16 of what hi leaves (22 bits together).
// Pads up to the pitch are zero.  Grid: (blocks over rows x pitch / 8, matrix),
// from the end to the start: the update that the pass before wrote last is still
// in L2.
template <bool kFp32, bool kVecOk>
__global__ void __launch_bounds__(kThreads) ns_scale_kernel(const __grid_constant__ ScaleArgs a) {
  __shared__ float power_shared, rest_shared;
  const int mat = static_cast<int>(gridDim.y - 1 - blockIdx.y);
  const long long block = gridDim.x - 1 - blockIdx.x;
  // The partials and the source are read once the pass before has finished; the
  // next kernel, another stack's momentum pass or the first product, may begin
  // once the last of these CTAs has got here.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // every CTA sums the matrix's partials, in the same order
  double s = 0.0;
  if (threadIdx.x < 32) {
    for (long long k = threadIdx.x; k < a.chunks; k += 32) s += a.partials[mat * a.chunks + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_down_sync(0xffffffffu, s, o);
  }
  if (threadIdx.x == 0) {
    // x scale / d.  Where 1 / d leaves fp32's range, by a power of two first, 2^100
    // or 2^-100: sqrt(s) reaches from 2^-149 to 2^148.
    const double d = sqrt(s) + a.eps;
    const float rough = static_cast<float>(d);
    if (rough >= 0x1p-60f && rough <= 0x1p60f) {
      power_shared = 1.0f;
      rest_shared = static_cast<float>(a.scale / d);
    } else {
      const float power = rough < 1.0f ? 0x1p100f : 0x1p-100f;
      power_shared = power;
      rest_shared = d == 0.0 ? 0.0f  // a zero matrix stays one without eps, too
                    : d <= 1e300 ? static_cast<float>(a.scale / (d * power)) : __int_as_float(0x7fffffff);
    }
  }
  __syncthreads();
  const float power = power_shared, rest = rest_shared;
  const long long vecs_per_row = a.ldx / kVec, total = a.rows * vecs_per_row;
  const bool small = total <= 0xffffffffLL;  // 32-bit divisions
  for (int i = 0; i < a.per_thread; ++i) {
    const long long v = (block * a.per_thread + i) * kThreads + threadIdx.x;
    if (v >= total) break;
    const long long row = small ? static_cast<uint32_t>(v) / static_cast<uint32_t>(vecs_per_row) : v / vecs_per_row;
    const long long col = (v - row * vecs_per_row) * kVec;
    const long long left = a.cols - col;
    const int count = static_cast<int>(left < 0 ? 0 : left < kVec ? left : kVec);
    float x[kVec];
    const long long at = mat * a.src.mat_stride + row * a.src.row_stride + col;
    if (kVecOk && count == kVec) {
      load8<kFp32, kVecOk>(a.src.data, at, count, x);
    } else {
      load8<kFp32, false>(a.src.data, at, count, x);
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float u = x[2 * k] * power * rest, w = x[2 * k + 1] * power * rest;
      const __half2 h = __floats2half2_rn(u, w);
      const __half2 l = __floats2half2_rn(u - __low2float(h), w - __high2float(h));
      hi[k] = *reinterpret_cast<const uint32_t*>(&h);
      lo[k] = *reinterpret_cast<const uint32_t*>(&l);
    }
    const long long to = (mat * a.rows + row) * a.ldx + col;
    *reinterpret_cast<uint4*>(a.hi + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (a.lo) *reinterpret_cast<uint4*>(a.lo + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

}  // namespace

cudaError_t launch_momentum(const MomentumArgs& a, bool vec, bool follows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.mats));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = follows ? 1 : 0;
  if (a.grad_fp32) {
    return vec ? cudaLaunchKernelEx(&cfg, momentum_kernel<true, true>, a)
               : cudaLaunchKernelEx(&cfg, momentum_kernel<true, false>, a);
  }
  return vec ? cudaLaunchKernelEx(&cfg, momentum_kernel<false, true>, a)
             : cudaLaunchKernelEx(&cfg, momentum_kernel<false, false>, a);
}

cudaError_t launch_ns_norm(const MatSource& s, const NsPlan& p, int mats, double* partials, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>(mats));
  const long long numel = p.rows * p.cols;
  if (s.fp32) {
    if (s.vec_ok) ns_norm_kernel<true, true><<<grid, kThreads, 0, stream>>>(s, p.cols, numel, p.chunks, partials);
    else ns_norm_kernel<true, false><<<grid, kThreads, 0, stream>>>(s, p.cols, numel, p.chunks, partials);
  } else {
    if (s.vec_ok) ns_norm_kernel<false, true><<<grid, kThreads, 0, stream>>>(s, p.cols, numel, p.chunks, partials);
    else ns_norm_kernel<false, false><<<grid, kThreads, 0, stream>>>(s, p.cols, numel, p.chunks, partials);
  }
  return cudaGetLastError();
}

cudaError_t launch_ns_scale(ScaleArgs a, cudaStream_t stream) {
  // What the GPU holds at once (8 CTAs per SM), or up to 16 vectors per thread,
  // so that the sum of the partials counts little.
  const long long work = a.rows * (a.ldx / kVec), room = 8LL * sm_count() * kThreads;
  const long long per = (work * a.mats + room - 1) / room;
  a.per_thread = static_cast<int>(per < 1 ? 1 : per < 16 ? per : 16);
  const long long block = static_cast<long long>(kThreads) * a.per_thread;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((work + block - 1) / block), static_cast<unsigned>(a.mats));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.src.fp32) {
    return a.src.vec_ok ? cudaLaunchKernelEx(&cfg, ns_scale_kernel<true, true>, a)
                        : cudaLaunchKernelEx(&cfg, ns_scale_kernel<true, false>, a);
  }
  return a.src.vec_ok ? cudaLaunchKernelEx(&cfg, ns_scale_kernel<false, true>, a)
                      : cudaLaunchKernelEx(&cfg, ns_scale_kernel<false, false>, a);
}

unsigned int muon_debug_failures() {
#ifdef ZFS_DEBUG_CHECKS
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_debug_failures, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
#else
  return 0;
#endif
}

}  // namespace zfs
