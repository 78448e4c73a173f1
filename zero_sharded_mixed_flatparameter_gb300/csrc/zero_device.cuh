// Device helpers shared by the step kernels and the auxiliary kernels of the
// ZeRO flat-parameter library: bf16 bit conversions, streaming (evict-first)
// 16-byte accesses and the grid-stride start index.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace zfs {

// Debug builds (-DZFS_DEBUG_CHECKS) check every index before the access it
// guards: a failed check counts in this file's counter and the access is
// skipped (no trap, no out-of-range access).  Release builds compile the
// checks away.
#ifdef ZFS_DEBUG_CHECKS
static __device__ unsigned int g_debug_failures = 0;
__device__ __forceinline__ bool debug_check(bool ok) {
  if (!ok) atomicAdd(&g_debug_failures, 1u);
  return ok;
}
#define ZFS_CHECK(cond) (::zfs::debug_check(static_cast<bool>(cond)))
#else
#define ZFS_CHECK(cond) true
#endif

__device__ __forceinline__ float bf16_lo(uint32_t word) { return __uint_as_float(word << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t word) { return __uint_as_float(word & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);  // .x = lo (low half), .y = hi
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint16_t to_bf16_bits(float x) {
  __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<uint16_t*>(&h);
}

// Streaming (evict-first) global accesses: every byte is touched once per step.
__device__ __forceinline__ uint4 ld_stream(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ float4 ld_stream_f4(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void st_stream_f4(float* p, float4 x) { __stcs(reinterpret_cast<float4*>(p), x); }
__device__ __forceinline__ void st_stream(void* p, uint4 x) { __stcs(reinterpret_cast<uint4*>(p), x); }

// A sum of squares in fp32 is taken as it is within these bounds.  Outside, or
// when it is NaN, the squares of finite entries may have over- or underflowed,
// and it is formed again from the entries times a power of two, kNormDown or
// kNormUp (every finite fp32 value, up to 2^37 of them, then stays in range).
constexpr float kNormLow = 0x1p-80f, kNormHigh = 0x1p100f, kNormUp = 0x1p90f, kNormDown = 0x1p-90f;

// Eight consecutive values from element `at` of a bf16 or fp32 array; kVecOk:
// the address is 16-byte aligned and all eight exist.
template <bool kFp32, bool kVecOk>
__device__ __forceinline__ void load8(const void* base, long long at, int count, float* x) {
  if constexpr (kVecOk) {
    if constexpr (kFp32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 u = p[0], v = p[1];
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf16_lo(w[k]);
        x[2 * k + 1] = bf16_hi(w[k]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = 0.0f;
      if (k < count) {
        if constexpr (kFp32) {
          x[k] = static_cast<const float*>(base)[at + k];
        } else {
          x[k] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at + k]) << 16);
        }
      }
    }
  }
}

// How many of kN reduced gradients are inf or NaN (the step's overflow
// count): one comparison and one add per value, no branch, so that the
// kernels' loads are not held behind it; the sum reaches the caller's counter
// only when counting is on (flush_nonfinite).
template <int kN>
__device__ __forceinline__ unsigned tally_nonfinite(const float* g) {
  unsigned c = 0;
#pragma unroll
  for (int e = 0; e < kN; ++e) c += (fabsf(g[e]) <= 0x1.fffffep127f) ? 0u : 1u;
  return c;
}

// Adds a thread's overflow count to the caller's counter (none when zero).
__device__ __forceinline__ void flush_nonfinite(unsigned long long* counter, unsigned count) {
  if (count != 0u && counter != nullptr) atomicAdd(counter, static_cast<unsigned long long>(count));
}

// First index >= 0 congruent to (tid - start) modulo stride: walking a
// segment from there in steps of `stride` makes the launch's grid-stride
// loop run over all segments as one concatenated index space.
__device__ __forceinline__ long long first_index(long long tid, long long start, long long stride) {
  long long r = (tid - start) % stride;
  return r < 0 ? r + stride : r;
}

}  // namespace zfs
