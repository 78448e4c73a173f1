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
// Bound by the tensor cores where the matrices are large: eight 2048-wide
// decoder layers run the last product of a step at 1.5 PFLOP/s (a 64-deep block
// of a pair's tile in 666 cycles, 512 at the nominal rate); by latency where
// they are small (a launch of one 512 x 2048 matrix takes 7.5 us, its products
// 2.3).
//
// One persistent CTA (or pair of CTAs on one tile, kCtas = 2) per SM.  Warp
// roles: 0-7 epilogue (TMEM quadrant warp % 4, column half warp / 4), 8 TMA
// loads, 9 issues the MMAs.  kStages stages of a 128 x 64 block of A and of B
// per CTA; two accumulators, so that the epilogue of a tile runs under the
// next one's products.  In a pair each CTA holds 128 of the 256 rows of A and
// half of B's columns, and the first CTA issues for both.
//
// Each epilogue warp works by itself, 32 rows by 64 columns at a time with its
// own 8 KB of shared memory.  The products leave little of shared memory's
// bandwidth (of 128 bytes a cycle, 64 go to loads and 64 to the MMAs at their
// peak), so the epilogue spares it: C (hi and lo) comes in by cp.async while
// the products still run, D goes out from registers, a 32-byte sector per lane
// and access, and only the transposed half of a symmetric tile crosses the
// buffer.  24 matrices of 1024 x 2048, five steps: 1054 us with C and D both by
// TMA through the buffer (their copies queue behind the operands'), 1010 so,
// 1152 with C read into registers as D is written.  The final update crosses
// the buffer so that master and param16 are read and written in whole rows.
// (Rows read and written by a thread each, 16 bytes at a time, cost the L1 a
// line per lane: 170 us for an update of 16 1024 x 2048 matrices whose products
// take 60; one buffer for all warps costs a barrier and a store's latency per 64
// columns: 16 products of 1024 took 61 us, 33 without any epilogue.)

#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "zero_device.cuh"
#include "zero_muon_internal.h"
#include "zero_tensor.cuh"

namespace zfs {
namespace {

constexpr int kBlockK = 64;            // fp16 elements of one 128-byte swizzled row
constexpr int kBlockM = 128;           // rows per CTA
constexpr int kStages = 5;
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = (kEpilogueWarps + 2) * 32;
constexpr uint32_t kOperandBytes = kBlockM * kBlockK * 2;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kChunk = 64;             // columns of a step of the epilogue
constexpr uint32_t kHalfBytes = 32 * kChunk * 2;  // a warp's chunk of hi (or of lo, or transposed)
constexpr uint32_t kBufferBytes = 2 * kHalfBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kEpilogueWarps * kBufferBytes + 1024;  // + alignment

// One stack of equal matrices.
struct Problem {
  CUtensorMap a, b;
  GemmArgs g;
  int first;                     // tile of the launch
  int tiles_m, tiles_n, tiles;   // tiles of one matrix
  int k_blocks;
  int vec_out;                   // kNsOut / kNsMuon: four elements of a row are aligned
};

// What one launch needs: stacks of several shapes share it, so that small ones
// do not leave the GPU to a few tiles at a time.
template <int kProblems>
struct GemmKernelArgs {
  Problem p[kProblems];
  int problems, total;           // tiles of all
};

// ---- epilogue ----------------------------------------------------------------
// Address of the 16-byte piece `piece` (of 8) of row r in a 32 x 64 half.
__device__ __forceinline__ uint32_t piece_at(uint32_t half, int r, int piece) {
  return half + r * 128 + ((piece ^ (r & 7)) << 4);
}

// A 32 x 64 half from global memory: 16 bytes per lane, four whole rows of 128
// bytes per access.  `rows` x `columns` of it lie inside the matrix, the rest
// reads as zero; whole pieces are read, up to the pitch.
__device__ __forceinline__ void load_half(uint32_t half, const uint16_t* from, long long pitch, long long rows,
                                          long long columns, int lane) {
  const int piece = lane % 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + lane / 8;
    const bool inside = r < rows && 8 * piece < columns;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(piece_at(half, r, piece)),
                 "l"(from + (inside ? r * pitch + 8 * piece : 0)), "r"(inside ? 16 : 0)
                 : "memory");
  }
}

// 16 fp16 of a row to global memory, a whole 32-byte sector per lane.
__device__ __forceinline__ void store_sector(uint16_t* to, const uint32_t* h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]),
               "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
               : "memory");
}

// Where column `lane` of row c of a transposed half (64 x 32, rows of 64 bytes)
// lies, and rows 8 k to 8 k + 7 of it to global memory.
__device__ __forceinline__ uint32_t mirror_at(uint32_t half, int c, int column) {
  return half + c * 64 + (((column / 8) ^ ((c >> 1) & 3)) << 4) + column % 8 * 2;
}
__device__ __forceinline__ void store_mirror(uint32_t half, int k, uint16_t* to, long long pitch, long long rows,
                                             long long columns, int lane) {
  const int r = 8 * k + lane / 4, piece = lane % 4;
  const uint4 v = lds16(mirror_at(half, r, 8 * piece));
  if (r < rows && 8 * piece < columns) *reinterpret_cast<uint4*>(to + r * pitch + 8 * piece) = v;
}

// y[0..31] += factor * 32 fp16 of row r, from piece `first`.
__device__ __forceinline__ void add_pieces(uint32_t half, int r, int first, float factor, float* y) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const uint4 h = lds16(piece_at(half, r, first + v));
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 u = half2_values(w[k]);
      y[8 * v + 2 * k] = fmaf(factor, u.x, y[8 * v + 2 * k]);
      y[8 * v + 2 * k + 1] = fmaf(factor, u.y, y[8 * v + 2 * k + 1]);
    }
  }
}

// Whole rows of a warp's finished chunk (32 x 64 fp32 in `buffer`, 16-byte
// pieces swizzled by row) to their place, from row i0 and column j0.
template <int kEpi>
__device__ __forceinline__ void store_rows(const Problem& p, int mat, uint32_t buffer, long long i0, long long j0,
                                           int lane) {
  const GemmArgs& g = p.g;
  const long long base = kEpi == kNsMuon ? g.out.offset[mat] : mat * g.out.mat_stride;
  const long long pitch = kEpi == kNsMuon ? g.N : g.out.row_stride;
  if (p.vec_out && j0 + kChunk <= g.N) {  // two rows per access
    const int piece = lane % 16;
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      float4 old[8];
      if constexpr (kEpi == kNsMuon) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = (q * 8 + k) * 2 + lane / 16;
          const long long at = base + (i0 + r) * pitch + j0 + 4 * piece;
          if (i0 + r < g.M && ZFS_CHECK(at >= 0 && at + 4 <= g.out.total_padded))
            old[k] = *reinterpret_cast<const float4*>(g.out.master + at);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = (q * 8 + k) * 2 + lane / 16;
        const long long at = base + (i0 + r) * pitch + j0 + 4 * piece;
        if (i0 + r >= g.M) continue;
        const uint4 v = lds16(buffer + r * 256 + ((piece ^ (r & 7)) << 4));
        float4 y = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
        if constexpr (kEpi == kNsMuon) {
          if (!ZFS_CHECK(at >= 0 && at + 4 <= g.out.total_padded)) continue;
          y.x = __fadd_rn(__fmul_rn(old[k].x, g.out.decay), __fmul_rn(-g.out.step, y.x));
          y.y = __fadd_rn(__fmul_rn(old[k].y, g.out.decay), __fmul_rn(-g.out.step, y.y));
          y.z = __fadd_rn(__fmul_rn(old[k].z, g.out.decay), __fmul_rn(-g.out.step, y.z));
          y.w = __fadd_rn(__fmul_rn(old[k].w, g.out.decay), __fmul_rn(-g.out.step, y.w));
          *reinterpret_cast<float4*>(g.out.master + at) = y;
          *reinterpret_cast<uint2*>(g.out.p16 + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        } else {
          *reinterpret_cast<uint2*>(g.out.out + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        }
      }
    }
  } else {  // columns lane and lane + 32
#pragma unroll 4
    for (int k = 0; k < 64; ++k) {
      const int r = k / 2, c = lane + 32 * (k % 2);
      if (i0 + r >= g.M || j0 + c >= g.N) continue;
      const long long at = base + (i0 + r) * pitch + j0 + c;
      float y;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(y)
                   : "r"(buffer + r * 256 + (((c / 4) ^ (r & 7)) << 4) + c % 4 * 4)
                   : "memory");
      if constexpr (kEpi == kNsMuon) {
        if (!ZFS_CHECK(at >= 0 && at < g.out.total_padded)) continue;
        y = __fadd_rn(__fmul_rn(g.out.master[at], g.out.decay), __fmul_rn(-g.out.step, y));
        g.out.master[at] = y;
        g.out.p16[at] = to_bf16_bits(y);
      } else {
        g.out.out[at] = to_bf16_bits(y);
      }
    }
  }
}

// Tile t of the launch: its stack, matrix, tile row and column.
struct Tile {
  int problem, mat, ti, tj;
};
template <int kEpi, int kProblems>
__device__ __forceinline__ Tile locate(const GemmKernelArgs<kProblems>& ka, int t) {
  Tile at;
  at.problem = 0;
  if constexpr (kProblems > 1) {
    while (at.problem + 1 < ka.problems && t >= ka.p[at.problem + 1].first) ++at.problem;
  }
  const Problem& p = ka.p[at.problem];
  t -= p.first;
  at.mat = t / p.tiles;
  int r = t - at.mat * p.tiles;
  if constexpr (kEpi == kNsGram || kEpi == kNsPoly) {  // rows of the lower triangle, one after another
    int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while (static_cast<long long>(i) * (i + 1) / 2 > r) --i;
    while (static_cast<long long>(i + 1) * (i + 2) / 2 <= r) ++i;
    at.ti = i;
    at.tj = r - static_cast<int>(static_cast<long long>(i) * (i + 1) / 2);
  } else {  // bands of 8 tile rows, so that tiles in flight share operands in L2
    constexpr int kBand = 8;
    const int band = r / (kBand * p.tiles_n), first = band * kBand;
    const int high = p.tiles_m - first < kBand ? p.tiles_m - first : kBand;
    r -= band * kBand * p.tiles_n;
    at.ti = first + r % high;
    at.tj = r / high;
  }
  return at;
}

template <int kCtas, int kEpi, int kProblems>
__global__ void __launch_bounds__(kGemmThreads, 1) ns_gemm_kernel(const __grid_constant__ GemmKernelArgs<kProblems> ka) {
  constexpr int kBlockN = 128 * kCtas;  // columns of a tile; rows: kBlockM * kCtas
  constexpr uint32_t kTmemColumns = 2 * kBlockN;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u, buffers = stages + kStages * kStageBytes;
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
  if (warp == 8) {  // the maps are there before the first copy asks for them
    for (int i = lane; i < 2 * ka.problems; i += 32)
      asm volatile("prefetch.tensormap [%0];" ::"l"(i % 2 ? &ka.p[i / 2].b : &ka.p[i / 2].a) : "memory");
  }
  if (warp == 9) tmem_alloc<kCtas>(smem_u32(&tmem_base), kTmemColumns);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas, total = ka.total;
  // The next kernel may take free SMs from here on; what the one before wrote
  // is read only after it has finished.
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool skip = false;
  if constexpr (kEpi == kNsMuon) skip = ka.p[0].g.out.dev_t && *ka.p[0].g.out.dev_t >= ka.p[0].g.out.dev_steps;

  if (warp == 8 && lane == 0 && !skip) {
    // ---- loads: both CTAs of a pair count on the first one's barrier ---------
    asm volatile("fence.proxy.async;" ::: "memory");  // what plain stores of the kernel before wrote
    uint32_t stage = 0, parity = 0;
    long long issued = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile at_tile = locate<kEpi>(ka, t);
      const Problem& p = ka.p[at_tile.problem];
      const int i0 = at_tile.ti * kBlockM * kCtas + rank * kBlockM, j0 = at_tile.tj * kBlockN + rank * 128;
      const int mat = at_tile.mat, k_steps = p.k_blocks;
      const bool a_k = p.g.a.k_major, b_k = p.g.b.k_major;
      for (int s = 0; s < k_steps; ++s) {
        const int k0 = s * kBlockK;
        if (!wait_phase(empty + 8 * stage, parity ^ 1, &gave_up)) {
          ok = false;
          break;
        }
        const uint32_t at = stages + stage * kStageBytes;
        const uint32_t bar = kCtas == 2 ? map_rank(full + 8 * stage, 0) : full + 8 * stage;
        if (rank == 0) mbar_expect_tx(full + 8 * stage, kStageBytes * kCtas);
        if (a_k) {
          tma_load<kCtas>(at, &p.a, k0, i0, mat, bar);
        } else {
          tma_load<kCtas>(at, &p.a, i0, k0, mat, bar);
          tma_load<kCtas>(at + kOperandBytes / 2, &p.a, i0 + 64, k0, mat, bar);
        }
        if (b_k) {
          tma_load<kCtas>(at + kOperandBytes, &p.b, k0, j0, mat, bar);
        } else {
          tma_load<kCtas>(at + kOperandBytes, &p.b, j0, k0, mat, bar);
          tma_load<kCtas>(at + kOperandBytes + kOperandBytes / 2, &p.b, j0 + 64, k0, mat, bar);
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
    uint32_t stage = 0, parity = 0, acc = 0, acc_parity = 0;
    bool ok = true;
    // What differs between stacks, looked up a tile ahead.
    bool a_k = true, b_k = true;
    int k_steps = 0;
    auto look_up = [&](int t, bool& a, bool& b, int& steps) {
      if (t >= total) return;
      const Problem& p = ka.p[locate<kEpi>(ka, t).problem];
      a = p.g.a.k_major;
      b = p.g.b.k_major;
      steps = p.k_blocks;
    };
    look_up(first, a_k, b_k, k_steps);
    for (int t = first; t < total && ok; t += step) {
      const uint32_t idesc = (1u << 4) | (a_k ? 0u : 1u << 15) | (b_k ? 0u : 1u << 16) |
                             (static_cast<uint32_t>(kBlockN >> 3) << 17) |
                             (static_cast<uint32_t>((kBlockM * kCtas) >> 4) << 24);
      const uint64_t step_a = a_k ? 32 >> 4 : 2048 >> 4, step_b = b_k ? 32 >> 4 : 2048 >> 4;
      bool next_a = true, next_b = true;
      int next_steps = 0;
      ok = wait_phase(tmem_empty + 8 * acc, acc_parity ^ 1, &gave_up);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + acc * kBlockN;
      for (int s = 0; s < k_steps; ++s) {
        ok = wait_phase(full + 8 * stage, parity, &gave_up);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t at = stages + stage * kStageBytes;
        const uint64_t da = smem_desc(at, a_k, 8192), db = smem_desc(at + kOperandBytes, b_k, 8192);
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k)
          mma<kCtas>(d, da + k * step_a, db + k * step_b, idesc, s > 0 || k > 0 ? 1 : 0);
        mma_commit<kCtas>(empty + 8 * stage);
        if (s == 0) look_up(t + step, next_a, next_b, next_steps);
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
      if (!ok) break;
      mma_commit<kCtas>(tmem_full + 8 * acc);
      a_k = next_a;
      b_k = next_b;
      k_steps = next_steps;
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
  } else if (warp < kEpilogueWarps && !skip) {
    // ---- epilogue -------------------------------------------------------------
    constexpr bool kHasC = kEpi != kNsGram;
    constexpr bool kRows = kEpi == kNsOut || kEpi == kNsMuon;  // finished rows
    constexpr bool kSymmetric = kEpi == kNsGram || kEpi == kNsPoly;
    constexpr int kChunks = kBlockN / kChunk / 2;  // per warp and tile
    const int quadrant = warp % 4, half = warp / 4;
    const uint32_t buffer = buffers + warp * kBufferBytes;
    const bool has_lo = ka.p[0].g.c_lo != nullptr, makes_lo = ka.p[0].g.d_lo != nullptr;  // as of every stack
    // This warp's C of a tile's chunk into its buffer.
    auto load_c = [&](int t, int chunk) {
      const Tile at = locate<kEpi>(ka, t);
      const GemmArgs& g = ka.p[at.problem].g;
      const long long i0 = at.ti * kBlockM * kCtas + rank * kBlockM + quadrant * 32;
      const long long j0 = static_cast<long long>(at.tj) * kBlockN + (2 * chunk + half) * kChunk;
      const bool some = i0 < g.M && j0 < g.N;
      const long long from = some ? at.mat * g.d_mat_stride + i0 * g.ldd + j0 : 0, rows = some ? g.M - i0 : 0;
      load_half(buffer, g.c + from, g.ldd, rows, g.N - j0, lane);
      if (has_lo) load_half(buffer + kHalfBytes, g.c_lo + from, g.ldd, rows, g.N - j0, lane);
    };
    uint32_t acc = 0, acc_parity = 0;
    if (kHasC && first < total) load_c(first, 0);
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile at = locate<kEpi>(ka, t);
      const Problem& p = ka.p[at.problem];
      const GemmArgs& g = p.g;
      const int mat = at.mat, ti = at.ti, tj = at.tj;
      const int i0 = ti * kBlockM * kCtas + rank * kBlockM + quadrant * 32;
      const bool mirror = kSymmetric && ti != tj;
      if constexpr (kEpi == kNsMuon) {
        // the tile's master rows on their way into L2 while the products run
        for (int chunk = 0; chunk < kChunks; ++chunk) {
          const long long j = static_cast<long long>(tj) * kBlockN + (2 * chunk + half) * kChunk;
          if (i0 + lane < g.M && j < g.N) {
            const float* w = g.out.master + g.out.offset[mat] + (i0 + lane) * g.N + j;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(w) : "memory");
            if (j + 32 < g.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + 32) : "memory");
          }
        }
      }
      ok = __all_sync(0xffffffffu, wait_phase(tmem_full + 8 * acc, acc_parity, &gave_up));
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
      for (int chunk = 0; chunk < kChunks; ++chunk) {
        const int j0 = tj * kBlockN + (2 * chunk + half) * kChunk;
        const uint32_t from = tmem + acc * kBlockN + ((quadrant * 32) << 16) + (2 * chunk + half) * kChunk;
        if constexpr (kHasC) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
        }
        float y[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_load32(from + 32 * q, y[q]);
#pragma unroll
          for (int k = 0; k < 32; ++k) y[q][k] *= g.alpha;
          if constexpr (kHasC) {
            add_pieces(buffer, lane, 4 * q, g.cfactor, y[q]);
            if (has_lo) add_pieces(buffer + kHalfBytes, lane, 4 * q, g.cfactor, y[q]);
          }
          if constexpr (!kRows) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const float* z = y[q] + 16 * v;
              const int c0 = 32 * q + 16 * v;
              const bool inside = i0 + lane < g.M && j0 + c0 < g.N;
              const long long to = mat * g.d_mat_stride + (i0 + lane) * g.ldd + j0 + c0;
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) h[k] = half2_bits(z[2 * k], z[2 * k + 1]);
              if (inside) store_sector(g.d + to, h);
              if constexpr (kEpi == kNsApply) {
                if (makes_lo) {
                  uint32_t l[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const float2 hv = half2_values(h[k]);
                    l[k] = half2_bits(z[2 * k] - hv.x, z[2 * k + 1] - hv.y);
                  }
                  if (inside) store_sector(g.d_lo + to, l);
                }
              } else if (mirror) {
                // transposed, rows of 64 bytes: row c, column `lane`
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  sts2(mirror_at(buffer + kHalfBytes, c0 + k, lane), static_cast<uint16_t>(h[k / 2] >> (16 * (k % 2))));
              }
            }
          }
        }
        if (chunk + 1 == kChunks) {  // this warp's part of the accumulator is drained
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(kCtas == 2 ? map_rank(tmem_empty + 8 * acc, 0) : tmem_empty + 8 * acc);
        }
        if constexpr (kRows) {
          __syncwarp();  // every lane has its C
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              sts16(buffer + lane * 256 + (((8 * q + v) ^ (lane & 7)) << 4),
                    make_uint4(__float_as_uint(y[q][4 * v]), __float_as_uint(y[q][4 * v + 1]),
                               __float_as_uint(y[q][4 * v + 2]), __float_as_uint(y[q][4 * v + 3])));
          }
          __syncwarp();
          if (i0 < g.M && j0 < g.N) store_rows<kEpi>(p, mat, buffer, i0, j0, lane);
        } else {
          __syncwarp();
          if (mirror && i0 < g.M && j0 < g.N) {
            uint16_t* to = g.d + mat * g.d_mat_stride + j0 * g.ldd + i0;
#pragma unroll
            for (int k = 0; k < 8; ++k) store_mirror(buffer + kHalfBytes, k, to, g.ldd, g.M - j0, g.N - i0, lane);
          }
        }
        __syncwarp();  // the buffer is free
        if constexpr (kHasC) {
          if (chunk + 1 < kChunks) load_c(t, chunk + 1);
          else if (t + step < total) load_c(t + step, 0);
        }
      }
      acc ^= 1;
      if (acc == 0) acc_parity ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (in flight only if a role gave up)
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 9) tmem_free<kCtas>(tmem, kTmemColumns);
}

// ---- few tiles, many k ---------------------------------------------------------
// A Gram matrix with so few tiles that most SMs would idle: a cluster of kSplit
// CTAs per tile, each over its share of k.  Every CTA leaves its sums (fp32) in
// its shared memory, and each joins a part of the tile from all of them, in
// rank order.  One 512 x 2048 matrix: the product over 32 blocks of k takes 9.4
// us in one CTA at the rate its operands come in; in eight, 2.3 us for 4 blocks
// each, 0.7 to put the sums down and meet, 2.3 to join them.
template <int kSplit>
__global__ void __launch_bounds__(kGemmThreads, 1) ns_gram_split_kernel(const __grid_constant__ GemmKernelArgs<1> ka) {
  constexpr int kUnits = 8 / kSplit;  // 32 x 64 parts of the tile that a CTA joins
  constexpr uint32_t kTmemColumns = 128;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const Problem& p = ka.p[0];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t stages = (smem_u32(smem_raw) + 1023) & ~1023u, buffers = stages + kStages * kStageBytes;
  const int rank = blockIdx.x % kSplit;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tmem_full = empty + 8 * kStages;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(tmem_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&p.a) : "memory");
  if (warp == 9) tmem_alloc<1>(smem_u32(&tmem_base), kTmemColumns);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Tile at = locate<kNsGram>(ka, blockIdx.x / kSplit);
  const int i0 = at.ti * kBlockM, j0 = at.tj * kBlockM;
  const int begin = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / kSplit);
  const int end = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / kSplit);
  const bool k_major = p.g.a.k_major;
  if (warp == 8 && lane == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");  // what plain stores of the kernel before wrote
    int issued = 0;
    bool ok = true;
    for (int s = begin; s < end && ok; ++s) {
      const int stage = issued % kStages;
      ok = wait_phase(empty + 8 * stage, issued / kStages & 1 ^ 1, &gave_up);
      if (!ok) break;
      const uint32_t to = stages + stage * kStageBytes, bar = full + 8 * stage;
      mbar_expect_tx(bar, kStageBytes);
      for (int operand = 0; operand < 2; ++operand) {
        const int x = operand ? j0 : i0;
        const uint32_t half = to + operand * kOperandBytes;
        if (k_major) {
          tma_load<1>(half, &p.a, s * kBlockK, x, at.mat, bar);
        } else {
          tma_load<1>(half, &p.a, x, s * kBlockK, at.mat, bar);
          tma_load<1>(half + kOperandBytes / 2, &p.a, x + 64, s * kBlockK, at.mat, bar);
        }
      }
      ++issued;
    }
    if (!ok) {  // a role gave up: the copies in flight land (bounded) before this CTA leaves
      const unsigned long long t0 = global_ns();
      for (bool landed = false; !landed && global_ns() - t0 < 50000000ull;) {
        landed = true;
        for (int s = 0; s < kStages; ++s) {
          const int uses = (issued + kStages - 1 - s) / kStages;
          if (uses > 0 && !mbar_try_wait(full + 8 * s, (uses - 1) & 1)) landed = false;
        }
      }
    }
  } else if (warp == 9 && lane == 0) {
    const uint32_t idesc = (1u << 4) | (k_major ? 0u : 3u << 15) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t step = k_major ? 32 >> 4 : 2048 >> 4;
    bool ok = true;
    for (int s = begin, n = 0; s < end; ++s, ++n) {
      const int stage = n % kStages;
      ok = wait_phase(full + 8 * stage, n / kStages & 1, &gave_up);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = stages + stage * kStageBytes;
      const uint64_t da = smem_desc(from, k_major, 8192), db = smem_desc(from + kOperandBytes, k_major, 8192);
#pragma unroll
      for (int k = 0; k < kBlockK / 16; ++k) mma<1>(tmem, da + k * step, db + k * step, idesc, n > 0 || k > 0 ? 1 : 0);
      mma_commit<1>(empty + 8 * stage);
    }
    if (ok) mma_commit<1>(tmem_full);
  } else if (warp < kEpilogueWarps) {
    // the sums to shared memory, where no stage is in use any more
    if (__all_sync(0xffffffffu, wait_phase(tmem_full, 0, &gave_up))) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t unit = stages + warp * 8192;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float y[32];
        tmem_load32(tmem + (((warp % 4) * 32) << 16) + warp / 4 * kChunk + 32 * q, y);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          sts16(unit + lane * 256 + (((8 * q + v) ^ (lane & 7)) << 4),
                make_uint4(__float_as_uint(y[4 * v]), __float_as_uint(y[4 * v + 1]), __float_as_uint(y[4 * v + 2]),
                           __float_as_uint(y[4 * v + 3])));
      }
    }
  }
  cluster_sync();
  if (warp < kEpilogueWarps) {
    const int mine = warp / kSplit, part = warp % kSplit, unit = rank * kUnits + mine;
    const uint32_t buffer = buffers + mine * kBufferBytes;
    const bool mirror = at.ti != at.tj;
    const long long i0 = at.ti * kBlockM + unit % 4 * 32, j0 = at.tj * kBlockM + unit / 4 * kChunk;
    uint16_t* d = p.g.d + at.mat * p.g.d_mat_stride;
#pragma unroll
    for (int q = 0; q < 16 / kSplit; ++q) {
      // a load takes two whole rows, 512 bytes in a line: the lanes' 16 bytes from
      // 32 rows took 6.6 us for the 64 KB
      const int row = 2 * (part * (16 / kSplit) + q) + lane / 16, piece = lane % 16;
      float y[4] = {};
#pragma unroll
      for (int r = 0; r < kSplit; ++r) {
        const float4 v = lds16_cluster(map_rank(stages + unit * 8192 + row * 256 + ((piece ^ (row & 7)) << 4), r));
        y[0] += v.x;
        y[1] += v.y;
        y[2] += v.z;
        y[3] += v.w;
      }
      uint32_t h[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) h[k] = half2_bits(y[2 * k] * p.g.alpha, y[2 * k + 1] * p.g.alpha);
      if (i0 + row < p.g.M && j0 + 4 * piece < p.g.N)
        *reinterpret_cast<uint2*>(d + (i0 + row) * p.g.ldd + j0 + 4 * piece) = make_uint2(h[0], h[1]);
      if (mirror) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 4 * piece + k;
          sts2(mirror_at(buffer, c, row), static_cast<uint16_t>(h[k / 2] >> (16 * (k % 2))));
        }
      }
    }
    if (mirror) {
      asm volatile("bar.sync 1, %0;" ::"n"(kEpilogueWarps * 32) : "memory");
#pragma unroll
      for (int k = part; k < 8; k += kSplit)
        store_mirror(buffer, k, d + j0 * p.g.ldd + i0, p.g.ldd, p.g.M - j0, p.g.N - i0, lane);
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // no CTA leaves while another reads its sums
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 9) tmem_free<1>(tmem, kTmemColumns);
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

// Launches `kernel` in clusters of `cluster` CTAs, after the kernel before it
// by programmatic serialization.
template <typename Args>
cudaError_t launch_clusters(void (*kernel)(const Args), const Args& ka, long long ctas, int cluster, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, ka);
}

template <int kCtas, int kEpi, int kProblems>
cudaError_t launch(GemmKernelArgs<kProblems>& ka, cudaStream_t stream) {
  const long long tile = 128 * kCtas;
  long long total = 0;
  for (int i = 0; i < ka.problems; ++i) {
    Problem& p = ka.p[i];
    const long long tiles_m = (p.g.M + tile - 1) / tile, tiles_n = (p.g.N + tile - 1) / tile;
    const long long all = kEpi == kNsGram || kEpi == kNsPoly ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n;
    if (total + all * p.g.mats > 0x3fffffffLL) return cudaErrorInvalidValue;
    p.first = static_cast<int>(total);
    p.tiles_m = static_cast<int>(tiles_m);
    p.tiles_n = static_cast<int>(tiles_n);
    p.tiles = static_cast<int>(all);
    total += all * p.g.mats;
  }
  ka.total = static_cast<int>(total);
  const long long room = sm_count() / kCtas;
  if constexpr (kCtas == 1 && kEpi == kNsGram && kProblems == 1) {
    // Clusters that the GPU holds at once, each CTA with at least 4 blocks of k.
    // (A cluster lies in one GPC: of 152 SMs, clusters of 8 reach 120 and of 4
    // reach 144.)  The five steps without and with it, us: 512 x 8192 325, 173;
    // 512 x 2048 165, 131; by four 896 x 2048 188, 156 and 512 x 1024 144, 127; by
    // two 1280 x 5120 342, 292 and 1100 x 1200 181, 173.
    const long long k_blocks = ka.p[0].k_blocks;
    if (total * 8 <= room * 3 / 4 && k_blocks >= 32)
      return launch_clusters(ns_gram_split_kernel<8>, ka, total * 8, 8, stream);
    if (total * 4 <= room * 15 / 16 && k_blocks >= 16)
      return launch_clusters(ns_gram_split_kernel<4>, ka, total * 4, 4, stream);
    if (total * 2 <= room && k_blocks >= 16) return launch_clusters(ns_gram_split_kernel<2>, ka, total * 2, 2, stream);
  }
  return launch_clusters(ns_gemm_kernel<kCtas, kEpi, kProblems>, ka, (total < room ? total : room) * kCtas, kCtas, stream);
}

template <int kEpi, int kProblems>
cudaError_t launch_tile(GemmKernelArgs<kProblems>& ka, cudaStream_t stream) {
  // A pair of SMs works on 256 x 256, one alone on 128 x 128.  A 64-deep block
  // takes both about as long (0.28 us: the pair's products, the single's
  // operands at 64 bytes a cycle), so the form that needs fewer rounds over the
  // GPU wins, give or take the longer epilogue of a pair (4 blocks).  Two Gram
  // matrices of 2048 x 8192: 97 us in singles (two rounds), 52 in pairs (one).
  auto cost = [&](long long tile, long long room) {
    long long tiles = 0, blocks = 0;
    for (int i = 0; i < ka.problems; ++i) {
      const Problem& p = ka.p[i];
      const long long m = (p.g.M + tile - 1) / tile, n = (p.g.N + tile - 1) / tile;
      const long long t = (kEpi == kNsGram || kEpi == kNsPoly ? m * (m + 1) / 2 : m * n) * p.g.mats;
      tiles += t;
      blocks += t * p.k_blocks;
    }
    const double mean = static_cast<double>(blocks) / static_cast<double>(tiles);
    return mean * static_cast<double>((tiles + room - 1) / room);
  };
  const int sms = sm_count();
  return cost(256, sms / 2) + 4.0 < cost(128, sms) ? launch<2, kEpi, kProblems>(ka, stream)
                                                   : launch<1, kEpi, kProblems>(ka, stream);
}

bool fill(const GemmArgs& g, Problem* p) {
  p->g = g;
  p->k_blocks = static_cast<int>((g.K + kBlockK - 1) / kBlockK);
  if (!encode(&p->a, g.a, g.M, g.K, g.mats) || !encode(&p->b, g.b, g.N, g.K, g.mats)) return false;
  p->vec_out = 0;
  if (g.epilogue == kNsOut) {
    p->vec_out = g.out.row_stride % 4 == 0 && g.out.mat_stride % 4 == 0 && reinterpret_cast<uintptr_t>(g.out.out) % 8 == 0;
  } else if (g.epilogue == kNsMuon) {
    p->vec_out = g.N % 4 == 0;
    for (int m = 0; m < g.mats; ++m) p->vec_out = p->vec_out && g.out.offset[m] % 4 == 0;
  }
  return true;
}

template <int kProblems>
cudaError_t launch_problems(const GemmArgs* g, int count, cudaStream_t stream) {
  GemmKernelArgs<kProblems> ka;
  ka.problems = count;
  // the deepest tiles first, so that the last round is of short ones
  int order[kProblems];
  for (int i = 0; i < count; ++i) order[i] = i;
  std::stable_sort(order, order + count, [&](int x, int y) { return g[x].K > g[y].K; });
  for (int i = 0; i < count; ++i)
    if (!fill(g[order[i]], &ka.p[i])) return cudaErrorInvalidValue;
  switch (g[0].epilogue) {
    case kNsGram: return launch_tile<kNsGram>(ka, stream);
    case kNsPoly: return launch_tile<kNsPoly>(ka, stream);
    case kNsApply: return launch_tile<kNsApply>(ka, stream);
    case kNsOut: return launch_tile<kNsOut>(ka, stream);
    default: return launch_tile<kNsMuon>(ka, stream);
  }
}

}  // namespace

cudaError_t launch_ns_gemm(const GemmArgs* g, int count, cudaStream_t stream, int* launches) {
  std::call_once(g_encode_once, load_encode);
  if (!g_encode) return cudaErrorNotSupported;
  ++*launches;
  // (a stack by itself spares the launch 12 KB of arguments)
  return count == 1 ? launch_problems<1>(g, count, stream) : launch_problems<kMaxProblems>(g, count, stream);
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
