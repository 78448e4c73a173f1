// The matrix products of the Newton-Schulz steps, on the tensor cores.
//
// A step on X (m x n over its smaller side m) is three products:
//   A = X X^T              symmetric: only tiles on and below the diagonal
//   P = b A + c A A        symmetric likewise
//   X' = a X + P X         the first term from X = hi + lo in the epilogue
// Operands are fp16 with a power-of-two scale, sums are fp32 in TMEM.  The
// identity stays out of P: its rounding on P's diagonal would dominate, and
// the low half of X, which matters for what the identity carries (directions
// that X all but lacks and later steps multiply by up to a), then needs no
// product of its own.  A tall G takes X^T X and X P instead, so that X keeps
// its orientation: operands whose inner (contiguous) index is the summed one
// are K-major, the others MN-major, and both are what the tensor cores read
// from shared memory.
//
// One persistent CTA (or pair of CTAs on one tile, kCtas = 2) per SM.  Warp
// roles: 0-7 epilogue (TMEM quadrant warp % 4, column half warp / 4), 8 TMA
// loads, 9 issues the MMAs.  kStages stages of a 128 x 64 block of A and of B
// per CTA; two accumulators, so that the epilogue of a tile runs under the
// next one's products.  In a pair each CTA holds 128 of the 256 rows of A and
// half of B's columns, and the first CTA issues for both.

#include <cuda.h>

#include <mutex>

#include "zero_device.cuh"
#include "zero_muon_internal.h"
#include "zero_tensor.cuh"

namespace zfs {
namespace {

constexpr int kBlockK = 64;            // fp16 elements of one 128-byte swizzled row
constexpr int kBlockM = 128;           // rows per CTA
constexpr int kStages = 6;
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = (kEpilogueWarps + 2) * 32;
constexpr uint32_t kOperandBytes = kBlockM * kBlockK * 2;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024;  // + alignment

// What one launch needs.
struct GemmKernelArgs {
  CUtensorMap a, b;
  GemmArgs g;
  long long tiles_m, tiles_n, tiles;  // tiles of one matrix / of all
  int k_blocks;
  int vec_out;                        // kNsOut / kNsMuon: 16-byte accesses allowed
};

// ---- epilogue ----------------------------------------------------------------
// x[0..7] += factor * the old iterate's 8 elements at `at`.
__device__ __forceinline__ void add_old(const GemmArgs& g, long long at, float* x) {
  const uint4 h = *reinterpret_cast<const uint4*>(g.c + at);
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = half2_values(hw[k]);
    x[2 * k] = fmaf(g.cfactor, v.x, x[2 * k]);
    x[2 * k + 1] = fmaf(g.cfactor, v.y, x[2 * k + 1]);
  }
  if (g.c_lo) {
    const uint4 l = *reinterpret_cast<const uint4*>(g.c_lo + at);
    const uint32_t lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = half2_values(lw[k]);
      x[2 * k] = fmaf(g.cfactor, v.x, x[2 * k]);
      x[2 * k + 1] = fmaf(g.cfactor, v.y, x[2 * k + 1]);
    }
  }
}

// 32 columns j .. j+31 of row i: x holds the sums.  `mirror`: an off-diagonal
// tile of a symmetric result, stored transposed as well (lanes are consecutive
// rows, so every column is one contiguous store of the warp).
template <int kEpi>
__device__ __forceinline__ void store_columns(const GemmKernelArgs& ka, int mat, long long i, long long j, bool mirror,
                                              float* x) {
  const GemmArgs& g = ka.g;
  if (i >= g.M || j >= g.N) return;
  // 8 columns at a time; the pitch of C and D is a multiple of 8
  const long long row = mat * g.d_mat_stride + i * g.ldd + j;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (j + 8 * v >= g.N) break;
    float* y = x + 8 * v;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= g.alpha;
    if constexpr (kEpi != kNsGram) add_old(g, row + 8 * v, y);
    if constexpr (kEpi == kNsGram || kEpi == kNsPoly || kEpi == kNsApply) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = half2_bits(y[2 * k], y[2 * k + 1]);
      *reinterpret_cast<uint4*>(g.d + row + 8 * v) = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (kEpi == kNsApply) {
        if (g.d_lo) {
          uint32_t l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 hv = half2_values(h[k]);
            l[k] = half2_bits(y[2 * k] - hv.x, y[2 * k + 1] - hv.y);
          }
          *reinterpret_cast<uint4*>(g.d_lo + row + 8 * v) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      } else if (mirror) {
        uint16_t* d = g.d + mat * g.d_mat_stride;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const long long c = j + 8 * v + k;
          if (c < g.N) d[c * g.ldd + i] = half_bits(y[k]);
        }
      }
    } else if constexpr (kEpi == kNsOut) {
      uint16_t* d = g.out.out + mat * g.out.mat_stride + i * g.out.row_stride + j + 8 * v;
      if (ka.vec_out && j + 8 * v + 8 <= g.N) {
        *reinterpret_cast<uint4*>(d) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                  pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (j + 8 * v + k < g.N) d[k] = to_bf16_bits(y[k]);
      }
    } else {
      const long long at = g.out.offset[mat] + i * g.N + j + 8 * v;
      float* w = g.out.master + at;
      uint16_t* p = g.out.p16 + at;
      if (ka.vec_out && j + 8 * v + 8 <= g.N) {
        if (!ZFS_CHECK(at >= 0 && at + 8 <= g.out.total_padded)) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 old = *reinterpret_cast<const float4*>(w + 4 * q);
          const float o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[4 * q + k] = __fadd_rn(__fmul_rn(o[k], g.out.decay), __fmul_rn(-g.out.step, y[4 * q + k]));
          *reinterpret_cast<float4*>(w + 4 * q) = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                  pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (j + 8 * v + k >= g.N || !ZFS_CHECK(at >= 0 && at + k < g.out.total_padded)) continue;
          const float z = __fadd_rn(__fmul_rn(w[k], g.out.decay), __fmul_rn(-g.out.step, y[k]));
          w[k] = z;
          p[k] = to_bf16_bits(z);
        }
      }
    }
  }
}

// Tile t of all matrices: (matrix, tile row, tile column).
template <int kEpi>
__device__ __forceinline__ void locate(const GemmKernelArgs& ka, long long t, int* mat, long long* ti, long long* tj) {
  *mat = static_cast<int>(t / ka.tiles);
  long long r = t - *mat * ka.tiles;
  if constexpr (kEpi == kNsGram || kEpi == kNsPoly) {  // rows of the lower triangle, one after another
    long long i = static_cast<long long>((sqrt(8.0 * static_cast<double>(r) + 1.0) - 1.0) * 0.5);
    while (i * (i + 1) / 2 > r) --i;
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    *ti = i;
    *tj = r - i * (i + 1) / 2;
  } else {  // bands of 8 tile rows, so that tiles in flight share operands in L2
    constexpr long long kBand = 8;
    const long long band = r / (kBand * ka.tiles_n), first = band * kBand;
    const long long high = ka.tiles_m - first < kBand ? ka.tiles_m - first : kBand;
    r -= band * kBand * ka.tiles_n;
    *ti = first + r % high;
    *tj = r / high;
  }
}

template <int kCtas, int kEpi>
__global__ void __launch_bounds__(kGemmThreads, 1) ns_gemm_kernel(const __grid_constant__ GemmKernelArgs ka) {
  constexpr int kBlockN = 128 * kCtas;  // columns of a tile; rows: kBlockM * kCtas
  constexpr uint32_t kTmemColumns = 2 * kBlockN;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const GemmArgs& g = ka.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t rank = kCtas == 2 ? blockIdx.x % 2 : 0;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tmem_full = empty + 8 * kStages,
                 tmem_empty = tmem_full + 16;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tmem_full + 8 * s, 1);
      mbar_init(tmem_empty + 8 * s, kEpilogueWarps * kCtas);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<kCtas>(smem_u32(&tmem_base), kTmemColumns);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  const long long first = blockIdx.x / kCtas, step = gridDim.x / kCtas, total = ka.tiles * g.mats;
  const int k_steps = ka.k_blocks;
  bool skip = false;
  if constexpr (kEpi == kNsMuon) skip = g.out.dev_t && *g.out.dev_t >= g.out.dev_steps;

  if (warp == 8 && lane == 0 && !skip) {
    // ---- loads: both CTAs of a pair count on the first one's barrier ---------
    uint32_t stage = 0, parity = 0;
    long long issued = 0;
    bool ok = true;
    for (long long t = first; t < total && ok; t += step) {
      int mat;
      long long ti, tj;
      locate<kEpi>(ka, t, &mat, &ti, &tj);
      const int i0 = static_cast<int>(ti * kBlockM * kCtas + rank * kBlockM);
      const int j0 = static_cast<int>(tj * kBlockN + rank * 128);
      for (int s = 0; s < k_steps; ++s) {
        const int k0 = s * kBlockK;
        if (!wait_phase(empty + 8 * stage, parity ^ 1, &gave_up)) {
          ok = false;
          break;
        }
        const uint32_t at = stages + stage * kStageBytes;
        const uint32_t bar = kCtas == 2 ? map_rank(full + 8 * stage, 0) : full + 8 * stage;
        if (rank == 0) mbar_expect_tx(full + 8 * stage, kStageBytes * kCtas);
        if (g.a.k_major) {
          tma_load<kCtas>(at, &ka.a, k0, i0, mat, bar);
        } else {
          tma_load<kCtas>(at, &ka.a, i0, k0, mat, bar);
          tma_load<kCtas>(at + kOperandBytes / 2, &ka.a, i0 + 64, k0, mat, bar);
        }
        if (g.b.k_major) {
          tma_load<kCtas>(at + kOperandBytes, &ka.b, k0, j0, mat, bar);
        } else {
          tma_load<kCtas>(at + kOperandBytes, &ka.b, j0, k0, mat, bar);
          tma_load<kCtas>(at + kOperandBytes + kOperandBytes / 2, &ka.b, j0 + 64, k0, mat, bar);
        }
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
    }
    // The MMAs' last arrivals reach this CTA's barriers before it may leave.
    for (int s = 0; s < kStages && ok && issued >= kStages; ++s) {
      ok = wait_phase(empty + 8 * stage, parity ^ 1, &gave_up);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
    for (int s = 0; s < issued && ok && issued < kStages; ++s) ok = wait_phase(empty + 8 * s, 0, &gave_up);
    if (!ok) {
      // a role gave up: the copies in flight land (bounded) before this CTA leaves
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < 50000000ull) {
        bool landed = true;
        if (rank == 0) {
          for (int s = 0; s < kStages; ++s) {
            // the phase of the last issue to this stage
            const long long uses = (issued + kStages - 1 - s) / kStages;
            if (uses > 0 && !mbar_try_wait(full + 8 * s, static_cast<uint32_t>((uses - 1) & 1))) landed = false;
          }
        } else {
          landed = false;  // the peer's copies count on the first CTA's barrier: wait the time out
        }
        if (landed) break;
      }
    }
  } else if (warp == 9 && lane == 0 && rank == 0 && !skip) {
    // ---- MMAs ---------------------------------------------------------------
    const uint32_t idesc = (1u << 4) | (g.a.k_major ? 0u : 1u << 15) | (g.b.k_major ? 0u : 1u << 16) |
                           (static_cast<uint32_t>(kBlockN >> 3) << 17) |
                           (static_cast<uint32_t>((kBlockM * kCtas) >> 4) << 24);
    const uint64_t step_a = g.a.k_major ? 32 >> 4 : 2048 >> 4, step_b = g.b.k_major ? 32 >> 4 : 2048 >> 4;
    uint32_t stage = 0, parity = 0, acc = 0, acc_parity = 0;
    bool ok = true;
    for (long long t = first; t < total && ok; t += step) {
      ok = wait_phase(tmem_empty + 8 * acc, acc_parity ^ 1, &gave_up);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + acc * kBlockN;
      for (int s = 0; s < k_steps; ++s) {
        ok = wait_phase(full + 8 * stage, parity, &gave_up);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t at = stages + stage * kStageBytes;
        const uint64_t da = smem_desc(at, g.a.k_major, 8192), db = smem_desc(at + kOperandBytes, g.b.k_major, 8192);
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k)
          mma<kCtas>(d, da + k * step_a, db + k * step_b, idesc, s > 0 || k > 0 ? 1 : 0);
        mma_commit<kCtas>(empty + 8 * stage);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
      if (!ok) break;
      mma_commit<kCtas>(tmem_full + 8 * acc);
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
  } else if (warp < kEpilogueWarps && !skip) {
    // ---- epilogue -------------------------------------------------------------
    const uint32_t quadrant = warp % 4, half = warp / 4;
    uint32_t acc = 0, acc_parity = 0;
    for (long long t = first; t < total; t += step) {
      int mat;
      long long ti, tj;
      locate<kEpi>(ka, t, &mat, &ti, &tj);
      if (!__all_sync(0xffffffffu, wait_phase(tmem_full + 8 * acc, acc_parity, &gave_up))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const long long i = ti * kBlockM * kCtas + rank * kBlockM + quadrant * 32 + lane;
      const bool mirror = (kEpi == kNsGram || kEpi == kNsPoly) && ti != tj;
#pragma unroll 1
      for (int c = half * kBlockN / 2; c < static_cast<int>(half + 1) * kBlockN / 2; c += 32) {
        float x[32];
        __syncwarp();
        tmem_load32(tmem + acc * kBlockN + ((quadrant * 32) << 16) + c, x);
        store_columns<kEpi>(ka, mat, i, tj * kBlockN + c, mirror, x);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(kCtas == 2 ? map_rank(tmem_empty + 8 * acc, 0) : tmem_empty + 8 * acc);
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 9) tmem_free<kCtas>(tmem, kTmemColumns);
}

// ---- host --------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeFn g_encode = nullptr;

void load_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess && fn) {
    g_encode = reinterpret_cast<EncodeFn>(fn);
  }
}

// Map of an operand with `mn` rows (columns) and `k` summed
// elements, read in boxes of 64 x 128 (K-major) or 64 x 64; what lies outside
// reads as zero.
bool encode(CUtensorMap* map, const GemmOperand& o, long long mn, long long k, int mats) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.k_major ? k : mn), static_cast<cuuint64_t>(o.k_major ? mn : k),
                              static_cast<cuuint64_t>(mats)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2, static_cast<cuuint64_t>(o.mat_stride) * 2};
  const cuuint32_t box[3] = {64, o.k_major ? 128u : 64u, 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(o.data), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCtas, int kEpi>
cudaError_t launch(GemmKernelArgs& ka, cudaStream_t stream) {
  const GemmArgs& g = ka.g;
  const long long tile = 128 * kCtas;
  ka.tiles_m = (g.M + tile - 1) / tile;
  ka.tiles_n = (g.N + tile - 1) / tile;
  ka.tiles = kEpi == kNsGram || kEpi == kNsPoly ? ka.tiles_m * (ka.tiles_m + 1) / 2 : ka.tiles_m * ka.tiles_n;
  const cudaError_t e =
      cudaFuncSetAttribute(ns_gemm_kernel<kCtas, kEpi>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const long long tiles = ka.tiles * g.mats, room = sm_count() / kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < room ? tiles : room) * kCtas));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ns_gemm_kernel<kCtas, kEpi>, ka);
}

template <int kEpi>
cudaError_t launch_tile(GemmKernelArgs& ka, cudaStream_t stream) {
  // A pair of SMs works on 256 x 256, one alone on 128 x 128: pairs once their
  // tiles fill the GPU.
  const long long t = 256;
  const long long m = (ka.g.M + t - 1) / t, n = (ka.g.N + t - 1) / t;
  const long long pairs = (kEpi == kNsGram || kEpi == kNsPoly ? m * (m + 1) / 2 : m * n) * ka.g.mats;
  return pairs >= sm_count() / 2 ? launch<2, kEpi>(ka, stream) : launch<1, kEpi>(ka, stream);
}

}  // namespace

cudaError_t launch_ns_gemm(const GemmArgs& g, cudaStream_t stream, int* launches) {
  std::call_once(g_encode_once, load_encode);
  if (!g_encode) return cudaErrorNotSupported;
  GemmKernelArgs ka;
  ka.g = g;
  ka.k_blocks = static_cast<int>((g.K + kBlockK - 1) / kBlockK);
  if (!encode(&ka.a, g.a, g.M, g.K, g.mats) || !encode(&ka.b, g.b, g.N, g.K, g.mats)) return cudaErrorInvalidValue;
  ka.vec_out = 0;
  if (g.epilogue == kNsOut) {
    ka.vec_out = g.out.row_stride % kVec == 0 && g.out.mat_stride % kVec == 0 &&
                 reinterpret_cast<uintptr_t>(g.out.out) % 16 == 0;
  } else if (g.epilogue == kNsMuon) {
    ka.vec_out = g.N % kVec == 0;
    for (int m = 0; m < g.mats; ++m) ka.vec_out = ka.vec_out && g.out.offset[m] % kVec == 0;
  }
  ++*launches;
  switch (g.epilogue) {
    case kNsGram: return launch_tile<kNsGram>(ka, stream);
    case kNsPoly: return launch_tile<kNsPoly>(ka, stream);
    case kNsApply: return launch_tile<kNsApply>(ka, stream);
    case kNsOut: return launch_tile<kNsOut>(ka, stream);
    default: return launch_tile<kNsMuon>(ka, stream);
  }
}

unsigned int ns_gemm_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
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
