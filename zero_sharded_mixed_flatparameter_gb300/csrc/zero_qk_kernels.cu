// Norm of the queries and keys of every head with the position rotation in
// the same pass, forward and backward, and their C calls.
//
//   y = x * rstd * gain,  rstd = 1 / sqrt(mean(x^2) + eps)
//   out = R(position) y   (R turns pairs of the first rotary_dim elements)
// backward, with xn = x * rstd and h = R^T dout:
//   dx = rstd * (gain h - xn * mean(gain h xn)),  dgain = sum h xn
//
// A head is read once and written once; everything between is fp32.  Bound by
// memory, so the kernel for heads of whole vectors keeps enough bytes in
// flight and instructions few: a group of lanes holds a head, two runs of 4
// elements a lane placed so that every rotated pair lies in one lane, a warp
// takes a token's heads kUnroll groups at a time, the token's cosines and sines
// stay in registers over its heads, the gains in shared memory, and addresses
// move by constant steps.  Other head sizes take one warp per head with the
// head in shared memory.
//
// 32768 tokens of 32 + 8 heads of 64, bf16: forward 55 us, 6.2 TB/s of the
// 344 MB read and written; backward 100 us, 5.1 TB/s of 512 MB (three streams
// with two reductions per head: its loads' latency counts, not the bandwidth),
// and 5 us for the gains' join.  5003 tokens of 16 + 4 heads of 80, fp32,
// backward: 26 + 5.5 us.

#include <cmath>
#include <cstdio>

#include "zero_device.cuh"
#include "zero_flatstep.h"
#include "zero_internal.h"
#include "zero_qk_internal.h"

namespace zfs {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kPerLane = kMaxHeadDim / 32;  // elements of a head per lane, at most

struct Heads {
  void* p;
  long long token, head;
};

struct QkArgs {
  long long tokens;
  int q_heads, k_heads, dim, rotary, interleaved;
  int gain_fp32, dgain_fp32;
  float eps;
  long long n_positions;
  Heads x[2], dy[2], out[2];   // queries, keys; out: the outputs or the inputs' gradients
  const void* gain[2];
  const float* table;
  const int32_t* positions;
  float* partials;             // [CTA][2][dim] gain sums of the backward pass
  void* dgain[2];
  int group;                   // lanes per head (power of two)
  int chunks, chunk_heads;     // a token's heads in parts for separate warps
};

template <bool kFp32>
__device__ __forceinline__ float load_one(const void* p, long long at) {
  if constexpr (kFp32) return static_cast<const float*>(p)[at];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at]) << 16);
}
template <bool kFp32>
__device__ __forceinline__ void store_one(void* p, long long at, float x) {
  if constexpr (kFp32) static_cast<float*>(p)[at] = x;
  else static_cast<uint16_t*>(p)[at] = to_bf16_bits(x);
}
__device__ __forceinline__ float load_gain(const QkArgs& a, int which, int d) {
  if (!a.gain[which]) return 1.0f;
  return a.gain_fp32 ? load_one<true>(a.gain[which], d) : load_one<false>(a.gain[which], d);
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The rotation of element d of the row in `row` (shared memory); `sign` +1
// turns, -1 turns back.
__device__ __forceinline__ float rotated(const QkArgs& a, const float* row, long long position, int d, float sign) {
  if (d >= a.rotary) return row[d];
  const int half = a.rotary / 2;
  const int pair = a.interleaved ? d / 2 : d % half;
  const bool first = a.interleaved ? d % 2 == 0 : d < half;
  const int other = a.interleaved ? d ^ 1 : first ? d + half : d - half;
  const float* t = a.table + position * a.rotary;
  const float cs = t[pair], sn = sign * t[half + pair];
  return first ? row[d] * cs - row[other] * sn : row[d] * cs + row[other] * sn;
}

template <bool kFp32, bool kBackward>
__global__ void __launch_bounds__(kQkThreads) qk_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float rows[kQkWarps][kMaxHeadDim];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float* row = rows[warp];
  const int heads = a.q_heads + a.k_heads;
  const long long total = a.tokens * heads;
  float dgain[2][kPerLane] = {};
  for (long long r = static_cast<long long>(blockIdx.x) * kQkWarps + warp; r < total;
       r += static_cast<long long>(gridDim.x) * kQkWarps) {
    const long long token = r / heads;
    const int h = static_cast<int>(r - token * heads), which = h < a.q_heads ? 0 : 1;
    const int head = which ? h - a.q_heads : h;
    const Heads &hx = a.x[which], &ho = a.out[which];
    const long long from = token * hx.token + head * hx.head, to = token * ho.token + head * ho.head;
    const long long position = a.positions ? a.positions[token] : token;
    if (position < 0 || position >= a.n_positions) {
      for (int d = lane; d < a.dim; d += 32) store_one<kFp32>(ho.p, to + d, 0.0f);
      continue;
    }
    float x[kPerLane] = {}, sq = 0.0f;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int d = lane + 32 * k;
      if (d < a.dim) x[k] = load_one<kFp32>(hx.p, from + d);
      sq += x[k] * x[k];
    }
    const float rstd = 1.0f / sqrtf(warp_sum(sq) / static_cast<float>(a.dim) + a.eps);
    __syncwarp();
    if constexpr (!kBackward) {
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int d = lane + 32 * k;
        if (d < a.dim) row[d] = x[k] * rstd * load_gain(a, which, d);
      }
      __syncwarp();
      for (int d = lane; d < a.dim; d += 32) store_one<kFp32>(ho.p, to + d, rotated(a, row, position, d, 1.0f));
    } else {
      const Heads& hy = a.dy[which];
      const long long at = token * hy.token + head * hy.head;
      for (int d = lane; d < a.dim; d += 32) row[d] = load_one<kFp32>(hy.p, at + d);
      __syncwarp();
      float g[kPerLane] = {}, dot = 0.0f;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int d = lane + 32 * k;
        if (d < a.dim) {
          const float t = rotated(a, row, position, d, -1.0f);
          x[k] *= rstd;
          if (which) dgain[1][k] += t * x[k];
          else dgain[0][k] += t * x[k];
          g[k] = t * load_gain(a, which, d);
          dot += g[k] * x[k];
        }
      }
      dot = warp_sum(dot) / static_cast<float>(a.dim);
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int d = lane + 32 * k;
        if (d < a.dim) store_one<kFp32>(ho.p, to + d, rstd * (g[k] - x[k] * dot));
      }
    }
  }
  if constexpr (kBackward) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) rows[warp][lane + 32 * k] = dgain[which][k];
      __syncthreads();
      for (int d = threadIdx.x; d < a.dim; d += kQkThreads) {
        float s = 0.0f;
        for (int w = 0; w < kQkWarps; ++w) s += rows[w][d];
        a.partials[(static_cast<long long>(blockIdx.x) * 2 + which) * a.dim + d] = s;
      }
    }
  }
}

// ---- heads of whole vectors --------------------------------------------------
// A lane's eight elements as loaded: two runs of 4.
template <bool kFp32>
struct Raw8 {
  uint32_t w[kFp32 ? 8 : 4];
};
template <bool kFp32, bool kAligned>
__device__ __forceinline__ void load4(const char* p, uint32_t* w) {
  if constexpr (kFp32 && kAligned) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (kFp32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = reinterpret_cast<const uint32_t*>(p)[k];
  } else if constexpr (kAligned) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] = static_cast<uint32_t>(q[2 * k]) | static_cast<uint32_t>(q[2 * k + 1]) << 16;
  }
}
// The lane's pairs: x[k] and x[4 + k] turn together.  Halves: elements k of
// the two runs; interleaved: neighbours.
template <bool kFp32>
__device__ __forceinline__ void widen(const Raw8<kFp32>& v, bool interleaved, float* x) {
  if constexpr (kFp32) {
    if (interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = __uint_as_float(v.w[2 * k]);
        x[4 + k] = __uint_as_float(v.w[2 * k + 1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(v.w[k]);
    }
  } else {
    if (interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = bf16_lo(v.w[k]);
        x[4 + k] = bf16_hi(v.w[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf16_lo(v.w[k]);
        x[2 * k + 1] = bf16_hi(v.w[k]);
      }
    }
  }
}
template <bool kFp32>
__device__ __forceinline__ void narrow(const float* x, bool interleaved, Raw8<kFp32>* v) {
  if constexpr (kFp32) {
    if (interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v->w[2 * k] = __float_as_uint(x[k]);
        v->w[2 * k + 1] = __float_as_uint(x[4 + k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v->w[k] = __float_as_uint(x[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v->w[k] = interleaved ? pack_bf16x2(x[k], x[4 + k]) : pack_bf16x2(x[2 * k], x[2 * k + 1]);
  }
}
template <bool kFp32, bool kAligned>
__device__ __forceinline__ void store4(char* p, const uint32_t* w) {
  if constexpr (kFp32 && kAligned) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (kFp32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<uint32_t*>(p)[k] = w[k];
  } else if constexpr (kAligned) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      q[2 * k] = static_cast<uint16_t>(w[k]);
      q[2 * k + 1] = static_cast<uint16_t>(w[k] >> 16);
    }
  }
}

// The lane's four pairs turned (kBack: turned back).
template <bool kBack>
__device__ __forceinline__ void turn(const float* cs, const float* sn, float* y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float one = y[k], two = y[4 + k], a = two * sn[k], b = one * sn[k];
    y[k] = fmaf(one, cs[k], kBack ? a : -a);
    y[4 + k] = fmaf(two, cs[k], kBack ? -b : b);
  }
}

// CTAs of the vector kernel on an SM: 32 warps forward (64 registers), 20
// backward (96).
constexpr int kVecThreads = 128, kVecWarps = kVecThreads / 32;
template <bool kBackward>
constexpr int kVecCtas = kBackward ? 5 : 8;

// kGroup: lanes per head, and aligned heads; 0: a.group lanes, any alignment.
template <bool kFp32, bool kBackward, int kGroup>
__global__ void __launch_bounds__(kVecThreads, kVecCtas<kBackward>)
    qk_vec_kernel(const __grid_constant__ QkArgs a) {
  constexpr int kThreads = kVecThreads, kWarps = kVecWarps;
  constexpr bool kAligned = kGroup != 0;
  constexpr int kUnroll = kBackward ? (kFp32 ? 1 : 2) : kFp32 ? 2 : 4;  // heads in flight per group of lanes
  constexpr long long kSize = kFp32 ? 4 : 2;
  // in the order of a lane's pairs: [query, key][lane of the group][8]
  __shared__ __align__(16) float gains[2][kMaxHeadDim];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = kGroup ? kGroup : a.group;
  const int in_group = lane % group, groups = 32 / group, my_group = lane / group;
  const int half = a.rotary / 2;
  const bool interleaved = a.interleaved != 0;
  const bool active = in_group * 8 < a.dim, turned = in_group * 8 < a.rotary;
  // the lane's two runs of 4 elements
  const int d0 = turned && !interleaved ? in_group * 4 : in_group * 8;
  const int d1 = turned && !interleaved ? half + in_group * 4 : in_group * 8 + 4;
  auto element = [&](int k) {  // of the lane's k-th value in pair order
    const int e = interleaved ? (k < 4 ? 2 * k : 2 * (k - 4) + 1) : k;
    return e < 4 ? d0 + e : d1 + e - 4;
  };
  if (warp == 0 && my_group == 0 && active) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int k = 0; k < 8; ++k) gains[which][in_group * 8 + k] = load_gain(a, which, element(k));
    }
  }
  __syncthreads();
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  const long long units = a.tokens * a.chunks, stride = static_cast<long long>(gridDim.x) * kWarps;
  auto position_of = [&](long long unit) -> long long {
    if (unit >= units) return -1;
    const long long token = a.chunks == 1 ? unit : unit / a.chunks;
    return a.positions ? a.positions[token] : token;
  };
  // Forward: a token's queries, then its keys.  Backward: all queries, then all
  // keys, so that one set of gain sums is live at a time.
#pragma unroll 1
  for (int pass = 0; pass < (kBackward ? 2 : 1); ++pass) {
  float dgain[8] = {};
  long long u = static_cast<long long>(blockIdx.x) * kWarps + warp;
  long long position = position_of(u);
  for (; u < units; u += stride) {
    const long long token = a.chunks == 1 ? u : u / a.chunks;
    const int begin = a.chunks == 1 ? 0 : static_cast<int>(u - token * a.chunks) * a.chunk_heads;
    const bool live = position >= 0 && position < a.n_positions;
    float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {};
    if (live && turned) {
      const float* row = a.table + position * a.rotary + in_group * 4;
      const float4 c = *reinterpret_cast<const float4*>(row);
      const float4 s = *reinterpret_cast<const float4*>(row + half);
      cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
      sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
    }
    position = position_of(u + stride);  // of the next token, while this one is worked on
#pragma unroll
    for (int part = 0; part < (kBackward ? 1 : 2); ++part) {
      const int which = kBackward ? pass : part;
      // the part of this unit's heads that are queries (keys)
      const int shift = which ? a.q_heads : 0, count = which ? a.k_heads : a.q_heads;
      const int lo = begin > shift ? begin - shift : 0;
      const int end = begin + a.chunk_heads - shift < count ? begin + a.chunk_heads - shift : count;
      if (lo >= end) continue;
      const Heads &hx = a.x[which], &hy = a.dy[which], &ho = a.out[which];
      const int mine = lo + my_group;
      const long long run = (d1 - d0) * kSize;
      const char* px = static_cast<const char*>(hx.p) + (token * hx.token + mine * hx.head + d0) * kSize;
      const char* py = kBackward ? static_cast<const char*>(hy.p) + (token * hy.token + mine * hy.head + d0) * kSize : nullptr;
      char* po = static_cast<char*>(ho.p) + (token * ho.token + mine * ho.head + d0) * kSize;
      const long long step_x = hx.head * groups * kSize, step_y = hy.head * groups * kSize, step_o = ho.head * groups * kSize;
      float gain[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 g = *reinterpret_cast<const float4*>(&gains[which][(active ? in_group * 8 : 0) + 4 * q]);
        gain[4 * q] = g.x; gain[4 * q + 1] = g.y; gain[4 * q + 2] = g.z; gain[4 * q + 3] = g.w;
      }
      int left = active ? end - mine : 0;  // heads from the lane's own on; > 0: it has one
#pragma unroll 1
      for (int h0 = lo; h0 < end; h0 += groups * kUnroll, left -= groups * kUnroll) {
        Raw8<kFp32> vx[kUnroll], vy[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          vx[i] = Raw8<kFp32>{};
          if constexpr (kBackward) vy[i] = Raw8<kFp32>{};
          if (left > i * groups) {
            load4<kFp32, kAligned>(px, vx[i].w);
            load4<kFp32, kAligned>(px + run, vx[i].w + (kFp32 ? 4 : 2));
            if constexpr (kBackward) {
              load4<kFp32, kAligned>(py, vy[i].w);
              load4<kFp32, kAligned>(py + run, vy[i].w + (kFp32 ? 4 : 2));
            }
          }
          px += step_x;
          if constexpr (kBackward) py += step_y;
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          if (h0 + i * groups >= end) break;  // the same for the whole warp
          const bool mine_too = left > i * groups;
          float x[8], y[8];
          widen<kFp32>(vx[i], interleaved, x);
          float sq = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) sq = fmaf(x[k], x[k], sq);
          if constexpr (!kBackward) {
#pragma unroll
            for (int o = group / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float rstd = rsqrtf(fmaf(sq, inv_dim, a.eps));
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = x[k] * rstd * gain[k];
            turn<false>(cs, sn, y);
          } else {
            widen<kFp32>(vy[i], interleaved, y);
            turn<true>(cs, sn, y);  // h: the gradient turned back
            float dot = 0.0f, g[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              g[k] = y[k] * gain[k];
              dot = fmaf(g[k], x[k], dot);
            }
#pragma unroll
            for (int o = group / 2; o > 0; o >>= 1) {
              sq += __shfl_xor_sync(0xffffffffu, sq, o);
              dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
            const float rstd = rsqrtf(fmaf(sq, inv_dim, a.eps));
            const float mean = dot * rstd * inv_dim;  // mean(gain h xn)
            const bool real = live && mine_too;       // else 0 * inf for eps 0, or what is behind padding
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float xn = x[k] * rstd;
              if (real) dgain[k] = fmaf(y[k], xn, dgain[k]);
              y[k] = rstd * fmaf(-xn, mean, g[k]);
            }
          }
          if (mine_too) {
            Raw8<kFp32> out;
            narrow<kFp32>(y, interleaved, &out);
            if (!live) out = Raw8<kFp32>{};
            store4<kFp32, kAligned>(po, out.w);
            store4<kFp32, kAligned>(po + run, out.w + (kFp32 ? 4 : 2));
          }
          po += step_o;
        }
      }
    }
  }
  if constexpr (kBackward) {
    // the CTA's gain sums: over the groups of a warp, then over the warps
    __shared__ float sums[kWarps][kMaxHeadDim];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      for (int o = group; o < 32; o <<= 1) dgain[k] += __shfl_xor_sync(0xffffffffu, dgain[k], o);
    }
    __syncthreads();
    if (my_group == 0 && active) {
#pragma unroll
      for (int k = 0; k < 8; ++k) sums[warp][element(k)] = dgain[k];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][d];
      a.partials[(static_cast<long long>(blockIdx.x) * 2 + pass) * a.dim + d] = s;
    }
  }
  }
}

// The gain gradients from the CTAs' sums: 32 columns per CTA, every warp a
// contiguous share of the CTAs, then warp after warp.  Launched so that it may
// become resident while the pass before it finishes; it waits for that pass.
constexpr int kGainThreads = 1024, kGainWarps = kGainThreads / 32;
__global__ void __launch_bounds__(kGainThreads) qk_gain_kernel(const __grid_constant__ QkArgs a, int ctas) {
  __shared__ float sums[kGainWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, column = blockIdx.x * 32 + lane;
  const int share = (ctas + kGainWarps - 1) / kGainWarps, begin = warp * share;
  const int end = begin + share < ctas ? begin + share : ctas;
  float s = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (column < 2 * a.dim) {
#pragma unroll 8
    for (int c = begin; c < end; ++c) s += a.partials[static_cast<long long>(c) * 2 * a.dim + column];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || column >= 2 * a.dim) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kGainWarps; ++w) s += sums[w][lane];
  const int which = column / a.dim;
  if (!a.dgain[which]) return;
  if (a.dgain_fp32) store_one<true>(a.dgain[which], column % a.dim, s);
  else store_one<false>(a.dgain[which], column % a.dim, s);
}

int next_power(int x) {
  int p = 1;
  while (p < x) p *= 2;
  return p;
}

// Whether heads fall into whole vectors of 8 for a lane.
bool lanes_ok(const QkArgs& a) {
  if (a.dim % 8) return false;
  if (a.rotary % 8) return false;
  return !a.rotary || reinterpret_cast<uintptr_t>(a.table) % 16 == 0;
}

// Whether all heads can then be read and written in one access a lane; the
// others go element by element with the same arithmetic.
bool vectors_ok(const QkArgs& a, bool fp32, bool backward) {
  const uintptr_t align = fp32 ? 16 : 8;
  for (int w = 0; w < 2; ++w) {
    if ((w ? a.k_heads : a.q_heads) == 0) continue;
    const Heads* all[3] = {&a.x[w], &a.out[w], backward ? &a.dy[w] : &a.x[w]};
    for (const Heads* h : all)
      if (reinterpret_cast<uintptr_t>(h->p) % align || h->token % 4 || h->head % 4) return false;
  }
  return true;
}

// CTAs of `warps` warps for `units` units of a warp's work, at most `per_sm` on an SM.
int qk_ctas(long long units, int warps, int per_sm) {
  const long long want = (units + warps - 1) / warps, most = static_cast<long long>(per_sm) * sm_count();
  return static_cast<int>(want < most ? want : most);
}
// The most that a backward launch over `rows` heads takes.
int backward_ctas(long long rows) {
  const int a = qk_ctas(rows, kQkWarps, 4), b = qk_ctas(rows, kVecWarps, kVecCtas<true>);
  return a > b ? a : b;
}

template <bool kFp32, bool kBackward>
int launch_qk(QkArgs& a, cudaStream_t s) {
  const long long rows = a.tokens * (a.q_heads + a.k_heads);
  int ctas = qk_ctas(rows, kQkWarps, 4);
  if (lanes_ok(a)) {
    // A warp takes a whole token while that gives every SM 16 warps (the
    // token's cosines are read once); fewer tokens are cut into parts.
    a.group = next_power(a.dim / 8);
    const int heads = a.q_heads + a.k_heads, groups = 32 / a.group;
    const long long most = (heads + groups - 1) / groups, wanted = 16LL * sm_count() / a.tokens;
    const long long parts = wanted < 1 ? 1 : wanted < most ? wanted : most;
    a.chunk_heads = static_cast<int>(((heads + parts - 1) / parts + groups - 1) / groups * groups);
    a.chunks = (heads + a.chunk_heads - 1) / a.chunk_heads;
    ctas = qk_ctas(a.tokens * a.chunks, kVecWarps, kVecCtas<kBackward>);
    const int group = vectors_ok(a, kFp32, kBackward) ? a.group : 0;
    switch (group) {
      case 4: qk_vec_kernel<kFp32, kBackward, 4><<<ctas, kVecThreads, 0, s>>>(a); break;
      case 8: qk_vec_kernel<kFp32, kBackward, 8><<<ctas, kVecThreads, 0, s>>>(a); break;
      case 16: qk_vec_kernel<kFp32, kBackward, 16><<<ctas, kVecThreads, 0, s>>>(a); break;
      case 32: qk_vec_kernel<kFp32, kBackward, 32><<<ctas, kVecThreads, 0, s>>>(a); break;
      default: qk_vec_kernel<kFp32, kBackward, 0><<<ctas, kVecThreads, 0, s>>>(a);
    }
  } else {
    qk_kernel<kFp32, kBackward><<<ctas, kQkThreads, 0, s>>>(a);
  }
  return ctas;
}

zero_status report(zero_status st, const char* text) {
  zfs_report_error(nullptr, st, text);
  return st;
}

// As the other calls of every step: NULL and alignment are checked, not where
// the memory lies (a query of the driver per pointer costs more than the
// launch of a single token's pass).
bool bad(const void* p, int esz) { return !p || reinterpret_cast<uintptr_t>(p) % esz != 0; }

zero_status check_config(const zero_qk_config* c, int64_t tokens) {
  if (!c) return report(ZERO_EINVAL, "config is NULL");
  if (tokens < 0) return report(ZERO_EINVAL, "tokens is negative");
  if (c->q_heads < 0 || c->k_heads < 0 || c->q_heads > (1 << 20) || c->k_heads > (1 << 20))
    return report(ZERO_EINVAL, "heads not in 0..2^20");
  if (c->head_dim < 2 || c->head_dim > kMaxHeadDim) return report(ZERO_EINVAL, "head_dim not in 2..256");
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 2)
    return report(ZERO_EINVAL, "rotary_dim must be even and in 0..head_dim");
  if (c->interleaved != 0 && c->interleaved != 1) return report(ZERO_EINVAL, "interleaved must be 0 or 1");
  if ((c->dtype != ZERO_GRAD_BF16 && c->dtype != ZERO_GRAD_FP32) ||
      (c->gain_dtype != ZERO_GRAD_BF16 && c->gain_dtype != ZERO_GRAD_FP32))
    return report(ZERO_EINVAL, "a dtype is neither bf16 (0) nor fp32 (1)");
  if (!(c->eps >= 0.0f) || !std::isfinite(c->eps)) return report(ZERO_EINVAL, "eps must be finite and >= 0");
  if (c->n_positions < 0) return report(ZERO_EINVAL, "n_positions is negative");
  return ZERO_OK;
}

// What both directions need; `tokens` > 0.
zero_status fill(const zero_qk_config* c, int64_t tokens, const zero_heads* q, const zero_heads* k, const void* q_gain,
                 const void* k_gain, const float* table, const int32_t* positions, const zero_heads* q_out,
                 const zero_heads* k_out, QkArgs* a) {
  const int esz = c->dtype == ZERO_GRAD_FP32 ? 4 : 2, gsz = c->gain_dtype == ZERO_GRAD_FP32 ? 4 : 2;
  const zero_heads* in[2] = {q, k};
  const zero_heads* out[2] = {q_out, k_out};
  const void* gain[2] = {q_gain, k_gain};
  const int heads[2] = {c->q_heads, c->k_heads};
  for (int w = 0; w < 2; ++w) {
    if (heads[w] == 0) continue;
    if (!in[w] || bad(in[w]->data, esz)) return report(ZERO_EINVAL, w ? "k is NULL or misaligned" : "q is NULL or misaligned");
    if (!out[w] || bad(out[w]->data, esz))
      return report(ZERO_EINVAL, w ? "k's output is NULL or misaligned" : "q's output is NULL or misaligned");
    if (in[w]->token_stride < 0 || in[w]->head_stride < 0 || out[w]->token_stride < 0 || out[w]->head_stride < 0)
      return report(ZERO_EINVAL, "a stride is negative");
    if (gain[w] && bad(gain[w], gsz)) return report(ZERO_EINVAL, "a gain is misaligned");
    a->x[w] = {in[w]->data, in[w]->token_stride, in[w]->head_stride};
    a->out[w] = {out[w]->data, out[w]->token_stride, out[w]->head_stride};
    a->gain[w] = gain[w];
  }
  if (c->rotary_dim > 0 && c->n_positions > 0 && bad(table, 4))
    return report(ZERO_EINVAL, "table is NULL or misaligned");
  if (positions && bad(positions, 4)) return report(ZERO_EINVAL, "positions is misaligned");
  a->tokens = tokens;
  a->q_heads = c->q_heads;
  a->k_heads = c->k_heads;
  a->dim = c->head_dim;
  a->rotary = c->rotary_dim;
  a->interleaved = c->interleaved;
  a->gain_fp32 = c->gain_dtype == ZERO_GRAD_FP32;
  a->eps = c->eps;
  a->n_positions = c->n_positions;
  a->table = table;
  a->positions = positions;
  return ZERO_OK;
}

zero_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return ZERO_OK;
  char buf[256];
  std::snprintf(buf, sizeof buf, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return report(ZERO_ECUDA, buf);
}

}  // namespace

unsigned int qk_debug_failures() {
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

zero_status zero_qk_norm_rope(const zero_qk_config* cfg, int64_t tokens, const zero_heads* q, const zero_heads* k,
                              const void* q_gain, const void* k_gain, const float* table, const int32_t* positions,
                              const zero_heads* q_out, const zero_heads* k_out, void* stream) {
  zero_status st = zfs::check_config(cfg, tokens);
  if (st != ZERO_OK) return st;
  if (tokens == 0 || cfg->q_heads + cfg->k_heads == 0) return ZERO_OK;
  zfs::QkArgs a{};
  st = zfs::fill(cfg, tokens, q, k, q_gain, k_gain, table, positions, q_out, k_out, &a);
  if (st != ZERO_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->dtype == ZERO_GRAD_FP32) zfs::launch_qk<true, false>(a, s);
  else zfs::launch_qk<false, false>(a, s);
  return zfs::launched("norm and rotation launch");
}

zero_status zero_qk_backward_workspace_bytes(const zero_qk_config* cfg, int64_t tokens, int64_t* bytes) {
  if (!bytes) return zfs::report(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_config(cfg, tokens);
  if (st != ZERO_OK) return st;
  *bytes = static_cast<int64_t>(zfs::backward_ctas(tokens * (cfg->q_heads + cfg->k_heads))) * 2 * cfg->head_dim * 4;
  return ZERO_OK;
}

zero_status zero_qk_norm_rope_backward(const zero_qk_config* cfg, int64_t tokens, const zero_heads* dq_out,
                                       const zero_heads* dk_out, const zero_heads* q, const zero_heads* k,
                                       const void* q_gain, const void* k_gain, const float* table,
                                       const int32_t* positions, const zero_heads* dq, const zero_heads* dk,
                                       void* dq_gain, void* dk_gain, int32_t dgain_dtype, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  zero_status st = zfs::check_config(cfg, tokens);
  if (st != ZERO_OK) return st;
  if (dgain_dtype != ZERO_GRAD_BF16 && dgain_dtype != ZERO_GRAD_FP32)
    return zfs::report(ZERO_EINVAL, "dgain_dtype is neither bf16 (0) nor fp32 (1)");
  const int dsz = dgain_dtype == ZERO_GRAD_FP32 ? 4 : 2;
  if ((dq_gain && zfs::bad(dq_gain, dsz)) || (dk_gain && zfs::bad(dk_gain, dsz)))
    return zfs::report(ZERO_EINVAL, "a gain gradient is misaligned");
  zfs::QkArgs a{};
  const long long rows = tokens * (cfg->q_heads + cfg->k_heads);
  int ctas = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    st = zfs::fill(cfg, tokens, q, k, q_gain, k_gain, table, positions, dq, dk, &a);
    if (st != ZERO_OK) return st;
    const zero_heads* dy[2] = {dq_out, dk_out};
    const int heads[2] = {cfg->q_heads, cfg->k_heads};
    for (int w = 0; w < 2; ++w) {
      if (heads[w] == 0) continue;
      if (!dy[w] || zfs::bad(dy[w]->data, cfg->dtype == ZERO_GRAD_FP32 ? 4 : 2))
        return zfs::report(ZERO_EINVAL, "an output gradient is NULL or misaligned");
      if (dy[w]->token_stride < 0 || dy[w]->head_stride < 0) return zfs::report(ZERO_EINVAL, "a stride is negative");
      a.dy[w] = {dy[w]->data, dy[w]->token_stride, dy[w]->head_stride};
    }
    int64_t need = 0;
    zero_qk_backward_workspace_bytes(cfg, tokens, &need);
    if (zfs::bad(workspace, 16)) return zfs::report(ZERO_EINVAL, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < need) return zfs::report(ZERO_EINVAL, "workspace is too small");
    a.partials = static_cast<float*>(workspace);
    ctas = cfg->dtype == ZERO_GRAD_FP32 ? zfs::launch_qk<true, true>(a, s) : zfs::launch_qk<false, true>(a, s);
    st = zfs::launched("norm and rotation backward launch");
    if (st != ZERO_OK) return st;
  }
  if (!dq_gain && !dk_gain) return ZERO_OK;
  a.dim = cfg->head_dim;
  a.dgain[0] = dq_gain;
  a.dgain[1] = dk_gain;
  a.dgain_fp32 = dgain_dtype == ZERO_GRAD_FP32;
  cudaLaunchConfig_t launch = {};
  launch.gridDim = dim3((2 * a.dim + 31) / 32);
  launch.blockDim = dim3(zfs::kGainThreads);
  launch.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  launch.attrs = attr;
  launch.numAttrs = 1;
  cudaLaunchKernelEx(&launch, zfs::qk_gain_kernel, a, ctas);
  return zfs::launched("gain gradient launch");
}

}  // extern "C"
