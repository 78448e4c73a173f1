// Device helpers of the kernels over rows of activations (layer norm, 8-bit
// form, embedding): eight elements of a row per thread, and the 8-bit codes.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "zero_device.cuh"

namespace zfs {

constexpr int kPackGroup = 32;                  // columns that share a scale
constexpr int kPackE4m3 = 1, kPackInt8 = 2;     // forms (0: none), as the public ones plus 1

// Two fp32 values in one register pair: the packed instructions round each like
// the single ones, at half the instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
__device__ __forceinline__ void split(F2 v, float* lo, float* hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v)); }
__device__ __forceinline__ float sum_of(F2 v) {
  float lo, hi;
  split(v, &lo, &hi);
  return lo + hi;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void to_pairs(const float* x, F2* p) {
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = pair(x[2 * k], x[2 * k + 1]);
}
__device__ __forceinline__ void from_pairs(const F2* p, float* x) {
#pragma unroll
  for (int k = 0; k < 4; ++k) split(p[k], &x[2 * k], &x[2 * k + 1]);
}

// Eight elements of a row as loaded.  kVec 8: eight neighbours from column
// 8 * lane on, 16-byte aligned; kVec 1: kCount (8, or fewer) columns lane,
// lane + lanes, ... (so that neighbouring threads read neighbouring columns
// whatever the alignment).
template <bool kFp32, int kVec, int kCount = 8>
struct Eight {
  uint32_t w[kVec == 1 ? kCount : kFp32 ? 8 : 4];
};

// The column of element k of thread `lane` of `lanes`, from column `first` on.
template <int kVec>
__device__ __forceinline__ int column(int k, int lane, int lanes) {
  return kVec == 8 ? lane * 8 + k : k * lanes + lane;
}

// How many of the thread's elements lie within `cols` columns are loaded; the
// others are zero.  `row`: the row's first element.
template <bool kFp32, int kVec, int kCount = 8>
__device__ __forceinline__ void load_eight(const void* row, int lane, int lanes, int cols, Eight<kFp32, kVec, kCount>* v) {
  if constexpr (kVec == 8) {
#pragma unroll
    for (int k = 0; k < (kFp32 ? 8 : 4); ++k) v->w[k] = 0u;
    if (lane * 8 < cols) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + static_cast<long long>(lane) * (kFp32 ? 32 : 16));
      const uint4 u = *p;
      v->w[0] = u.x; v->w[1] = u.y; v->w[2] = u.z; v->w[3] = u.w;
      if constexpr (kFp32) {
        const uint4 t = p[1];
        v->w[4] = t.x; v->w[5] = t.y; v->w[6] = t.z; v->w[7] = t.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int c = k * lanes + lane;
      v->w[k] = 0u;
      if (c < cols) {
        if constexpr (kFp32) v->w[k] = static_cast<const uint32_t*>(row)[c];
        else v->w[k] = static_cast<const uint16_t*>(row)[c];
      }
    }
  }
}

template <bool kFp32, int kVec, int kCount = 8>
__device__ __forceinline__ void widen_eight(const Eight<kFp32, kVec, kCount>& v, float* x) {
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    if constexpr (kFp32) x[k] = __uint_as_float(v.w[k]);
    else if constexpr (kVec == 8) x[k] = k % 2 ? bf16_hi(v.w[k / 2]) : bf16_lo(v.w[k / 2]);
    else x[k] = bf16_lo(v.w[k]);
  }
}

// Eight neighbours of a row at any alignment: single loads, of which a line's
// later ones find it in L1.
template <bool kFp32>
__device__ __forceinline__ void load_neighbours(const void* row, int lane, int cols, Eight<kFp32, 8>* v) {
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = lane * 8 + k;
    u[k] = 0u;
    if (c < cols) {
      if constexpr (kFp32) u[k] = static_cast<const uint32_t*>(row)[c];
      else u[k] = static_cast<const uint16_t*>(row)[c];
    }
  }
#pragma unroll
  for (int k = 0; k < (kFp32 ? 8 : 4); ++k) v->w[k] = kFp32 ? u[k] : u[2 * k] | u[2 * k + 1] << 16;
}
// A warp's 256 neighbours to a row at any alignment, turned in shared memory so
// that every store writes 32 neighbours.  `cols`: of the warp's.
template <bool kFp32>
__device__ __forceinline__ void store_neighbours(void* row, int cols, const F2* p, float* turned) {
  const int lane = threadIdx.x % 32;
  F2* mine = reinterpret_cast<F2*>(turned) + lane * 4;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) mine[k] = p[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = k * 32 + lane;
    if (c < cols) {
      if constexpr (kFp32) static_cast<float*>(row)[c] = turned[c];
      else static_cast<uint16_t*>(row)[c] = to_bf16_bits(turned[c]);
    }
  }
}

// Asynchronous copies of a thread's own bytes to its own place in shared memory:
// it waits for its own groups of copies, with no barrier and nothing to poll.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Widened anew where it is used again: eight fp32 values kept instead take twice
// the registers of the loaded words (bf16), four times those of codes.
template <typename T>
__device__ __forceinline__ void forget_widened(T& v) {
#pragma unroll
  for (uint32_t& w : v.w) asm volatile("" : "+r"(w));
}

template <bool kFp32, int kVec, int kCount = 8>
__device__ __forceinline__ void store_eight(void* row, int lane, int lanes, int cols, const float* x) {
  if constexpr (kVec == 8) {
    if (lane * 8 < cols) {
      uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(row) + static_cast<long long>(lane) * (kFp32 ? 32 : 16));
      if constexpr (kFp32) {
        p[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        p[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
      } else {
        p[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int c = k * lanes + lane;
      if (c < cols) {
        if constexpr (kFp32) static_cast<float*>(row)[c] = x[k];
        else static_cast<uint16_t*>(row)[c] = to_bf16_bits(x[k]);
      }
    }
  }
}

template <bool kFp32, int kVec>
__device__ __forceinline__ void widen_pairs(const Eight<kFp32, kVec>& v, F2* p) {
  float x[8];
  widen_eight<kFp32, kVec>(v, x);
  to_pairs(x, p);
}
template <bool kFp32, int kVec>
__device__ __forceinline__ void store_pairs(void* row, int lane, int lanes, int cols, const F2* p) {
  float x[8];
  from_pairs(p, x);
  store_eight<kFp32, kVec>(row, lane, lanes, cols, x);
}

// Element `at` of a bf16 or fp32 vector (weights, biases, their gradients).
__device__ __forceinline__ float load_scalar(const void* p, bool fp32, long long at) {
  if (fp32) return static_cast<const float*>(p)[at];
  return bf16_lo(static_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void store_scalar(void* p, bool fp32, long long at, float x) {
  if (fp32) static_cast<float*>(p)[at] = x;
  else static_cast<uint16_t*>(p)[at] = to_bf16_bits(x);
}

// ---- the 8-bit form ---------------------------------------------------------
// The byte of a group's scale 2^(byte - 127): the smallest power of two under
// which the group's largest magnitude (its fp32 bits) is at most 448 (e4m3) or
// 127 (int8).  A power of two scales without rounding, so that an element is
// rounded once; the e4m3 grid is the same under any of them but for what it
// underflows, and int8 gives up half a bit on average for it.  255: the group
// holds an inf or NaN; its codes are zero, and 0 * 2^128 (inf) reads as NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t largest, int form) {
  const uint32_t e = largest >> 23, m = largest & 0x7FFFFFu;
  if (e == 255u) return 255u;
  const int b = form == kPackE4m3 ? static_cast<int>(e) - 8 + (m > 0x600000u) : static_cast<int>(e) - 6 + (m > 0x7E0000u);
  return b < 1 ? 1u : static_cast<uint32_t>(b);
}
// 1 / scale (not for byte 255, whose codes are zero whatever the elements).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four elements (already times the inverse scale) as four codes, and back.
__device__ __forceinline__ uint32_t encode4(const float* x, int form) {
  if (form == kPackE4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) w |= (static_cast<uint32_t>(__float2int_rn(x[k])) & 0xFFu) << (8 * k);
  return w;
}
__device__ __forceinline__ void decode4(uint32_t w, int form, float* x) {
  if (form == kPackE4m3) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * k)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  } else {
    // a byte below an fp32 exponent of 2^23: 2^23 + 128 + code, exactly
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u + k)) - 8388736.0f;
  }
}
__device__ __forceinline__ uint32_t encode1(float x, int form) {
  if (form == kPackE4m3) return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(__float2int_rn(x)) & 0xFFu;
}
__device__ __forceinline__ float decode1(uint32_t code, int form) {
  if (form == kPackE4m3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return static_cast<float>(static_cast<int8_t>(code));
}

// The codes of the thread's eight neighbours, a quarter of a group whose others
// the next lanes hold, and the group's scale; every lane of the warp calls it.
// quarters: lanes that hold a part of the group (the rest of it does not exist).
__device__ __forceinline__ uint2 encode_eight(const F2* p, int quarters, int form, uint32_t* byte) {
  float x[8];
  from_pairs(p, x);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, m, o);
    if (o < quarters) m = max(m, other);
  }
  *byte = scale_byte(m, form);
  const F2 inv = both(inverse_scale(*byte));
  F2 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) q[k] = mul2(p[k], inv);
  from_pairs(q, x);
  return *byte == 255u ? make_uint2(0u, 0u) : make_uint2(encode4(x, form), encode4(x + 4, form));
}

// Writes the 8-bit form of the thread's eight neighbours (from column 8 * lane
// on); every lane of the warp calls it.  `lanes`: threads that hold the row (a
// power of two below 32, or a multiple of 32); `write`: the thread's row exists.
// Codes past the last column of the last group are zero.
__device__ __forceinline__ void pack_eight(const F2* p, int lane, int lanes, int groups, bool write, int form,
                                           uint8_t* codes, uint8_t* scales) {
  uint32_t byte;
  const uint2 c = encode_eight(p, lanes < 4 ? lanes : 4, form, &byte);
  if (write && lane < groups * 4) {
    *reinterpret_cast<uint2*>(codes + static_cast<long long>(lane) * 8) = c;
    if (lane % 4 == 0) scales[lane / 4] = static_cast<uint8_t>(byte);
    // fewer lanes than a group's quarters: the rest of the only group
    if (lanes < 4 && lane + 1 == lanes) {
      for (int q = lanes; q < 4; ++q) *reinterpret_cast<uint2*>(codes + q * 8) = make_uint2(0u, 0u);
    }
  }
}

// Single elements (column k * lanes + lane) are turned within the warp, in its
// 256 floats of shared memory, into eight neighbours of one of its eight groups of
// 32 columns, and back.
__device__ __forceinline__ void to_neighbours(const F2* singles, float* turned, F2* p) {
  const int l = threadIdx.x % 32;
  float x[8];
  from_pairs(singles, x);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) turned[k * 32 + l] = x[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = reinterpret_cast<const F2*>(turned)[l * 4 + k];
}
__device__ __forceinline__ void to_singles(const F2* p, float* turned, F2* singles) {
  const int l = threadIdx.x % 32;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) reinterpret_cast<F2*>(turned)[l * 4 + k] = p[k];
  __syncwarp();
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = turned[k * 32 + l];
  to_pairs(x, singles);
}
// The group of the n-th eight single elements whose neighbours this thread then has.
__device__ __forceinline__ int turned_group(int n, int lane, int lanes) {
  return (n * 8 + lane % 32 / 4) * (lanes / 32) + lane / 32;
}

// The thread's eight neighbours in 8 bits, as loaded, and as values.
struct EightCodes {
  uint32_t w[3];  // codes, the scale's byte
};
__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, int lane, int groups, EightCodes* v) {
  v->w[0] = v->w[1] = v->w[2] = 0u;
  if (lane < groups * 4) {
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(codes + static_cast<long long>(lane) * 8));
    v->w[0] = c.x; v->w[1] = c.y;
    v->w[2] = scales[lane / 4];
  }
}
__device__ __forceinline__ void widen_codes(const EightCodes& v, int form, F2* p) {
  float x[8];
  const F2 s = both(scale_value(v.w[2]));
  decode4(v.w[0], form, x);
  decode4(v.w[1], form, x + 4);
  to_pairs(x, p);
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = mul2(p[k], s);
}

}  // namespace zfs
