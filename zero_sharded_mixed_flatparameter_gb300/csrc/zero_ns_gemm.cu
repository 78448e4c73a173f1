// The matrix products of the Newton-Schulz steps.
//
// A step on X (m x n over its smaller side m) is three products:
//   A = X X^T            symmetric: only tiles on and below the diagonal
//   P = a I + b A + c A A  symmetric likewise
//   X' = P X             X = hi + lo while the early steps amplify rounding
// Operands are fp16 with a power-of-two scale, sums are fp32.

#include <cuda_fp16.h>

#include "zero_device.cuh"
#include "zero_muon_internal.h"

namespace zfs {
namespace {

constexpr int kTile = 64, kDepth = 16, kGemmThreads = 256;

__device__ __forceinline__ float half_bits(uint16_t b) {
  __half_raw r;
  r.x = b;
  return __half2float(__half(r));
}
__device__ __forceinline__ uint16_t to_half_bits(float x) {
  const __half h = __float2half_rn(x);
  return *reinterpret_cast<const uint16_t*>(&h);
}

// One element of the finished product at (i, j) of matrix `mat`.
__device__ __forceinline__ void store_one(const GemmArgs& g, int mat, long long i, long long j, float acc) {
  const float v = acc * g.alpha;
  if (g.epilogue == kNsGram || g.epilogue == kNsPoly) {
    uint16_t* d = g.d + mat * g.d_mat_stride;
    float x = v;
    if (g.epilogue == kNsPoly) {
      x = g.cc * v + g.cb * half_bits(g.c[mat * g.d_mat_stride + i * g.ldd + j]) + (i == j ? g.ca : 0.0f);
    }
    const uint16_t h = to_half_bits(x * g.out_scale);
    d[i * g.ldd + j] = h;
    d[j * g.ldd + i] = h;
  } else if (g.epilogue == kNsApply) {
    const float x = v * g.out_scale;
    const uint16_t h = to_half_bits(x);
    g.d[mat * g.d_mat_stride + i * g.ldd + j] = h;
    if (g.d_lo) g.d_lo[mat * g.d_mat_stride + i * g.ldd + j] = to_half_bits(x - half_bits(h));
  } else if (g.epilogue == kNsOut) {
    g.out.out[mat * g.out.mat_stride + i * g.out.row_stride + j] = to_bf16_bits(v);
  } else {
    const long long at = g.out.offset[mat] + i * g.N + j;
    if (!ZFS_CHECK(at >= 0 && at < g.out.total_padded)) return;
    const float w = __fadd_rn(__fmul_rn(g.out.master[at], g.out.decay), __fmul_rn(-g.out.step, v));
    g.out.master[at] = w;
    g.out.p16[at] = to_bf16_bits(w);
  }
}

template <bool kAK, bool kBK>
__global__ void __launch_bounds__(kGemmThreads) ns_gemm_kernel(const __grid_constant__ GemmArgs g) {
  __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
  if (g.epilogue == kNsMuon && g.out.dev_t && *g.out.dev_t >= g.out.dev_steps) return;
  const long long tiles_n = (g.N + kTile - 1) / kTile;
  const long long i0 = blockIdx.x / tiles_n * kTile, j0 = blockIdx.x % tiles_n * kTile;
  const bool symmetric = g.epilogue == kNsGram || g.epilogue == kNsPoly;
  if (symmetric && j0 > i0) return;
  const int mat = blockIdx.y, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int part = 0; part < g.parts; ++part) {
    const uint16_t* pa = g.a.part[part] + mat * g.a.mat_stride;
    const uint16_t* pb = g.b.part[part] + mat * g.b.mat_stride;
    for (long long k0 = 0; k0 < g.K; k0 += kDepth) {
      for (int e = threadIdx.x; e < kTile * kDepth; e += kGemmThreads) {
        {
          const int i = kAK ? e / kDepth : e % kTile, k = kAK ? e % kDepth : e / kTile;
          const bool in = i0 + i < g.M && k0 + k < g.K;
          as[k][i] = in ? half_bits(kAK ? pa[(i0 + i) * g.a.ld + k0 + k] : pa[(k0 + k) * g.a.ld + i0 + i]) : 0.0f;
        }
        {
          const int j = kBK ? e / kDepth : e % kTile, k = kBK ? e % kDepth : e / kTile;
          const bool in = j0 + j < g.N && k0 + k < g.K;
          bs[k][j] = in ? half_bits(kBK ? pb[(j0 + j) * g.b.ld + k0 + k] : pb[(k0 + k) * g.b.ld + j0 + j]) : 0.0f;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = as[k][ty + 16 * r];
          y[r] = bs[k][tx + 16 * r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(x[r], y[c], acc[r][c]);
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const long long i = i0 + ty + 16 * r, j = j0 + tx + 16 * c;
      if (i >= g.M || j >= g.N || (symmetric && j > i)) continue;
      store_one(g, mat, i, j, acc[r][c]);
    }
  }
}

}  // namespace

cudaError_t launch_ns_gemm(const GemmArgs& g, cudaStream_t stream, int* launches) {
  const dim3 grid(static_cast<unsigned>((g.N + kTile - 1) / kTile * ((g.M + kTile - 1) / kTile)),
                  static_cast<unsigned>(g.mats));
  if (g.a.k_major && g.b.k_major) ns_gemm_kernel<true, true><<<grid, kGemmThreads, 0, stream>>>(g);
  else if (g.a.k_major) ns_gemm_kernel<true, false><<<grid, kGemmThreads, 0, stream>>>(g);
  else ns_gemm_kernel<false, false><<<grid, kGemmThreads, 0, stream>>>(g);
  ++*launches;
  return cudaGetLastError();
}

unsigned int ns_gemm_debug_failures() {
#ifdef ZFS_DEBUG_CHECKS
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_debug_failures, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
#else
  return 0;
#endif
}

}  // namespace zfs
