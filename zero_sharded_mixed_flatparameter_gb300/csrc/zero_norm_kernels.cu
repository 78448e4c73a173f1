// Layer norm over the columns of a matrix, forward and backward, with the
// input's 8-bit form written and read in the same passes, and its C calls.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd weight + bias
// (mean 0 without centring).  Backward, with xn = (x - mean) rstd, g = dy weight:
//   dx = rstd (g - sum g / n - xn sum (g xn) / n),  dweight = sum dy xn,
//   dbias = sum dy
// (without the sum of g alone where nothing was centred).
//
// Every element is read once and written once, so memory is the floor; what has to
// be kept out of its way are the reductions and the instructions.  Forward: whole
// warps hold a row as loaded (up to 2048 bf16 columns a warp, so that most rows
// need no barrier) and widen it three times; the mean comes before the squares,
// which lose nothing to a far mean.  Backward: a thread keeps the same columns
// of all its rows, for the sums of dweight and dbias in registers, so a row takes
// more warps and a barrier; its rows are copied ahead to shared memory.  One CTA an
// SM, so that the column sums come in 152 parts.  Arithmetic is packed (two fp32 an
// instruction): both passes were bound by instructions without.
//
// Device times.  32768 x 2048 bf16, weight and bias: forward 46 us, 5.9 TB/s of the
// 268 MB read and written; backward 67 us, 6.0 TB/s of 403 MB, 3 of them the join
// of the column sums.  16384 x 2048 with the 8-bit form (e4m3), both directions: 74
// us for 338 MB.  There neither memory (42 % in use) nor issue slots (56 % forward,
// 65 % backward) are full: 16 to 20 warps an SM, a quarter of what it holds, convert
// codes between the sums they wait for; the backward pass decodes twice, and sums
// dbias and a mean of g that the form without them does not need.  16384 x 2048
// fp32: 46 us forward, 105 backward (268, 403 MB).  Widths that are no multiple of
// 8 columns go as single elements, with fewer rows in flight: 5003 x 1301 fp32 14
// us forward, 24 backward (52, 78 MB); 32768 x 2047 bf16 forward 78 us.  Beyond
// 8192 columns a CTA walks over the row: 4096 x 8192 bf16 32 us forward, 50
// backward, 4096 x 8200 97 and 122.

#include <cmath>

#include "zero_flatstep.h"
#include "zero_rows.cuh"
#include "zero_rows_host.h"

namespace zfs {
namespace {

constexpr int kLaneThreads = 256, kLaneCtas = 3;  // of the kernels that hold several rows in a warp, CTAs an SM
constexpr int kLaneCols = 128;                    // columns of a row of theirs, at most
// Warps of a CTA, one an SM: 96 registers a thread forward (16, 20 and 24 warps:
// 49, 46 and 47 us for 32768 x 2048), 128 backward.
constexpr int kForwardWarps = 20, kBackwardWarps = 16, kNormWarps = 20;
constexpr int kNormWidest = 8192;                 // columns that warps hold in registers
constexpr int kWideThreads = 512;                 // threads of a CTA that walks over a row

struct NormArgs {
  long long rows;
  int cols, lanes;           // lanes: threads that hold a row
  float inv_cols, eps;
  const void *x, *dy;        // x: NULL where the backward pass reads the 8-bit form
  void* out;                 // y, or dx
  long long x_stride, dy_stride, out_stride;
  const void *weight, *bias;
  int weight_fp32, center, want_bias;
  int form;                  // of the 8-bit form, 0: none
  int groups;                // a row's groups of 32 columns; its codes have 32 * groups bytes
  uint8_t *codes, *scales;
  float2* stats;             // mean, rstd of every row; NULL allowed forward
  float* partials;           // [part][dweight, dbias][cols]
  void *dweight, *dbias;
  int dgrad_fp32, parts;
};

// ---- rows of up to kLaneCols columns: a power of two of a warp's lanes each ------
template <int kN>
__device__ __forceinline__ void lanes_sum(float (&v)[kN], int lanes) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (o < lanes) {
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
}

__device__ __forceinline__ void load_vector(const void* p, bool fp32, int lane, int cols, float other, float* w) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = lane * 8 + k;
    w[k] = p && c < cols ? load_scalar(p, fp32, c) : other;
  }
}

template <bool kFp32>
__global__ void __launch_bounds__(kLaneThreads, kLaneCtas) norm_lanes_forward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = 2;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kLaneThreads / lanes;
  float w[8], b[8];
  load_vector(a.weight, a.weight_fp32, lane, a.cols, 1.0f, w);
  load_vector(a.bias, a.weight_fp32, lane, a.cols, 0.0f, b);
  const long long step = static_cast<long long>(gridDim.x) * per_cta, first = static_cast<long long>(blockIdx.x) * per_cta;
  // all threads take the same number of turns
  for (long long r0 = first; r0 < a.rows; r0 += step * kRows) {
    const long long mine = r0 + threadIdx.x / lanes;
    Eight<kFp32, 8> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + step * i;
      load_eight<kFp32, 8>(static_cast<const char*>(a.x) + r * a.x_stride * kSize, lane, lanes, r < a.rows ? a.cols : 0,
                           &raw[i]);
    }
    float x[kRows][8], mean[kRows] = {}, total[kRows] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      widen_eight<kFp32, 8>(raw[i], x[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) mean[i] += x[i][k];
    }
    if (a.center) lanes_sum(mean, lanes);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      mean[i] = a.center ? mean[i] * a.inv_cols : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = x[i][k] - mean[i];
        total[i] = fmaf(d, d, total[i]);
      }
      if (lane * 8 >= a.cols) total[i] = 0.0f;
    }
    lanes_sum(total, lanes);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + step * i;
      const bool real = r < a.rows;
      if (a.form != 0) {
        F2 pairs[4];
        to_pairs(x[i], pairs);
        pack_eight(pairs, lane, lanes, a.groups, real, a.form, a.codes + r * a.groups * kPackGroup,
                      a.scales + r * a.groups);
      }
      const float rstd = rsqrtf(fmaf(total[i], a.inv_cols, a.eps));
      if (a.stats && real && lane == 0) a.stats[r] = make_float2(mean[i], rstd);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = fmaf((x[i][k] - mean[i]) * rstd, w[k], b[k]);
      if (real) {
        store_eight<kFp32, 8>(static_cast<char*>(a.out) + r * a.out_stride * kSize, lane, lanes, a.cols, x[i]);
      }
    }
  }
}

// kPacked: x comes from its 8-bit form.
template <bool kFp32, bool kPacked>
__global__ void __launch_bounds__(kLaneThreads, kLaneCtas) norm_lanes_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = 2;
  constexpr long long kSize = kFp32 ? 4 : 2;
  const int lanes = a.lanes, lane = threadIdx.x % lanes, per_cta = kLaneThreads / lanes;
  float w[8], dw[8] = {}, db[8] = {};
  load_vector(a.weight, a.weight_fp32, lane, a.cols, 1.0f, w);
  const long long step = static_cast<long long>(gridDim.x) * per_cta, first = static_cast<long long>(blockIdx.x) * per_cta;
  const bool column = lane * 8 < a.cols;
  for (long long r0 = first; r0 < a.rows; r0 += step * kRows) {
    const long long mine = r0 + threadIdx.x / lanes;
    Eight<kFp32, 8> raw[kRows], grad[kRows];
    EightCodes codes[kRows];
    float2 stats[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + step * i;
      const bool real = r < a.rows;
      stats[i] = real ? a.stats[r] : make_float2(0.0f, 0.0f);
      if constexpr (kPacked) {
        load_codes(a.codes + r * a.groups * kPackGroup, a.scales + r * a.groups, lane, real ? a.groups : 0, &codes[i]);
      } else {
        load_eight<kFp32, 8>(static_cast<const char*>(a.x) + r * a.x_stride * kSize, lane, lanes, real ? a.cols : 0, &raw[i]);
      }
      load_eight<kFp32, 8>(static_cast<const char*>(a.dy) + r * a.dy_stride * kSize, lane, lanes, real ? a.cols : 0, &grad[i]);
    }
    float xn[kRows][8], g[kRows][8], total[2 * kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kPacked) {
        F2 pairs[4];
        widen_codes(codes[i], a.form, pairs);
        from_pairs(pairs, xn[i]);
      } else {
        widen_eight<kFp32, 8>(raw[i], xn[i]);
      }
      widen_eight<kFp32, 8>(grad[i], g[i]);
      total[2 * i] = total[2 * i + 1] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // columns past the last: nothing of the mean, of the row's inf or NaN
        xn[i][k] = column ? (xn[i][k] - stats[i].x) * stats[i].y : 0.0f;
        dw[k] = fmaf(g[i][k], xn[i][k], dw[k]);
        db[k] += g[i][k];
        g[i][k] *= w[k];
        total[2 * i] += g[i][k];
        total[2 * i + 1] = fmaf(g[i][k], xn[i][k], total[2 * i + 1]);
      }
    }
    lanes_sum(total, lanes);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + step * i;
      if (r >= a.rows) continue;
      const float m1 = a.center ? total[2 * i] * a.inv_cols : 0.0f, m2 = total[2 * i + 1] * a.inv_cols;
#pragma unroll
      for (int k = 0; k < 8; ++k) g[i][k] = stats[i].y * fmaf(-xn[i][k], m2, g[i][k] - m1);
      store_eight<kFp32, 8>(static_cast<char*>(a.out) + r * a.out_stride * kSize, lane, lanes, a.cols, g[i]);
    }
  }
  if (!a.partials) return;
  // over the groups of a warp, then over the warps
  __shared__ float sums[2][kLaneThreads / 32][kLaneCols];
  float* part = a.partials + static_cast<long long>(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    for (int o = lanes; o < 32; o <<= 1) {
      dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
      db[k] += __shfl_xor_sync(0xffffffffu, db[k], o);
    }
    if (threadIdx.x % 32 < lanes) {
      sums[0][threadIdx.x / 32][lane * 8 + k] = dw[k];
      sums[1][threadIdx.x / 32][lane * 8 + k] = db[k];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.cols; c += kLaneThreads) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float s = 0.0f;
      for (int v = 0; v < kLaneThreads / 32; ++v) s += sums[which][v][c];
      part[which * a.cols + c] = s;
    }
  }
}

// ---- rows of up to kNormWidest columns: whole warps each -------------------------
// A CTA's warps form groups of a.lanes threads, a group takes kRows rows at a
// time, a thread kN times eight columns of each.  The weights stand in shared
// memory in the order in which a thread reads them.
template <int kVec, int kN>
struct Slots {
  int lanes, lane;  // of the group
  // The n-th eight columns: from column `at`, as thread `lane_of` of the group.
  __device__ __forceinline__ int at(int n) const { return kVec == 8 ? 0 : n * 8 * lanes; }
  __device__ __forceinline__ int lane_of(int n) const { return kVec == 8 ? n * lanes + lane : lane; }
  __device__ __forceinline__ int column_of(int n, int k) const {
    return kVec == 8 ? (n * lanes + lane) * 8 + k : (n * 8 + k) * lanes + lane;
  }
  // Where a column's weight stands: the lower and the upper four of a thread's
  // eight apart, for 16-byte reads without conflicts.
  __device__ __forceinline__ int slot(int c) const {
    return kVec == 8 ? ((c % 8 / 4) * kN * lanes + c / 8) * 4 + c % 4 : c;
  }
  __device__ __forceinline__ void read(const float* table, int n, F2* w) const {
    if constexpr (kVec == 8) {
      const ulonglong2* t = reinterpret_cast<const ulonglong2*>(table) + n * lanes + lane;
      const ulonglong2 u = t[0], v = t[kN * lanes];
      w[0] = u.x; w[1] = u.y; w[2] = v.x; w[3] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pair(table[(n * 8 + 2 * k) * lanes + lane], table[(n * 8 + 2 * k + 1) * lanes + lane]);
    }
  }
  // Columns 4 * four .. 4 * four + 3 of a vector; those that do not exist: zero.
  __device__ __forceinline__ float4 load_four(const void* p, bool fp32, int four, int cols, float other) const {
    const int c = four * 4;
    float v[4];
    if (p && c + 4 <= cols && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      if (fp32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c);
      return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k >= cols ? 0.0f : p ? load_scalar(p, fp32, c + k) : other;
    return make_float4(v[0], v[1], v[2], v[3]);
  }
  // All the CTA's threads.
  __device__ __forceinline__ void store_four(float* table, int four, float4 v) const {
    *reinterpret_cast<float4*>(table + slot(four * 4)) = v;  // four neighbours in either order
  }
};

// Sums of kV values over the group's threads.
template <int kV>
struct GroupSum {
  float (*buffer)[kNormWarps][kV];  // [turn][warp of the CTA]
  int first, warps, barrier, turn;  // the group's first warp, how many, its barrier
  __device__ __forceinline__ GroupSum(float (*b)[kNormWarps][kV], int lanes)
      : buffer(b), first(threadIdx.x / lanes * (lanes / 32)), warps(lanes / 32), barrier(1 + threadIdx.x / lanes), turn(0) {}
  __device__ __forceinline__ void operator()(float (&v)[kV]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if (warps == 1) return;
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int i = 0; i < kV; ++i) buffer[turn][threadIdx.x / 32][i] = v[i];
    }
    // two alternating buffers: one barrier a sum is enough
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = 0.0f;
    for (int w = first; w < first + warps; ++w) {
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] += buffer[turn][w][i];
    }
    turn ^= 1;
  }
};

// Rows in flight, by the registers that a thread's part of one takes.
template <bool kFp32, int kVec, int kN>
constexpr int kForwardRows = kN * (kFp32 || kVec == 1 ? 2 : 1) >= 8 ? 1 : kN * (kFp32 || kVec == 1 ? 2 : 1) >= 4 ? 2 : 4;

// kForm: of the 8-bit form, 0: none.
template <bool kFp32, int kVec, int kN, int kForm>
__global__ void __launch_bounds__(kForwardWarps * 32, 1) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = kForwardRows<kFp32, kVec, kN>;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  extern __shared__ __align__(16) float tables[];
  __shared__ float buffer[2][kNormWarps][kRows];
  __shared__ __align__(16) float turned[kVec == 1 && kForm ? kForwardWarps : 1][256];
  GroupSum<kRows> sum(buffer, a.lanes);
  const Slots<kVec, kN> own{a.lanes, static_cast<int>(threadIdx.x) % a.lanes};
  float *weight = tables, *bias = tables + kN * 8 * a.lanes;
  const int groups = blockDim.x / a.lanes, group = threadIdx.x / a.lanes;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  // the first rows of the CTAs before their second ones
  const long long mine = blockIdx.x + static_cast<long long>(gridDim.x) * group;
  bool staged = false;
  for (long long r0 = mine; r0 < a.rows || !staged; r0 += step * kRows) {
    Eight<kFp32, kVec> raw[kRows][kN];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = r0 + step * i;
      const char* row = static_cast<const char*>(a.x) + r * a.x_stride * kSize;
#pragma unroll
      for (int n = 0; n < kN; ++n)
        load_eight<kFp32, kVec>(row + own.at(n) * kSize, own.lane_of(n), own.lanes, r < a.rows ? a.cols - own.at(n) : 0,
                                &raw[i][n]);
    }
    if (!staged) {  // while the first rows are on their way
      for (int four = threadIdx.x; four < kN * 2 * a.lanes; four += blockDim.x) {
        const float4 w = own.load_four(a.weight, a.weight_fp32, four, a.cols, 1.0f);
        const float4 b = own.load_four(a.bias, a.weight_fp32, four, a.cols, 0.0f);
        own.store_four(weight, four, w);
        own.store_four(bias, four, b);
      }
      __syncthreads();
      staged = true;
      if (r0 >= a.rows) break;
    }
    float mean[kRows] = {}, total[kRows] = {};
    if (a.center) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        F2 s = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          F2 x[4];
          widen_pairs<kFp32, kVec>(raw[i][n], x);
          s = add2(s, add2(add2(x[0], x[1]), add2(x[2], x[3])));
        }
        mean[i] = sum_of(s);
      }
      sum(mean);
    }
    F2 less[kRows];  // minus the mean
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      mean[i] *= a.inv_cols;
      less[i] = both(-mean[i]);
      F2 s = 0;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        F2 x[4], part = 0;
        forget_widened(raw[i][n]);
        widen_pairs<kFp32, kVec>(raw[i][n], x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          F2 d = add2(x[k], less[i]);
          if constexpr (kVec == 1) {
            float lo, hi;
            split(d, &lo, &hi);
            d = pair(own.column_of(n, 2 * k) < a.cols ? lo : 0.0f, own.column_of(n, 2 * k + 1) < a.cols ? hi : 0.0f);
          }
          part = fma2(d, d, part);
        }
        if (kVec == 8 && own.column_of(n, 0) >= a.cols) part = 0;
        s = add2(s, part);
      }
      total[i] = sum_of(s);
    }
    sum(total);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = r0 + step * i;
      const bool real = r < a.rows;
      const float rstd = rsqrtf(fmaf(total[i], a.inv_cols, a.eps));
      if (a.stats && real && own.lane == 0) a.stats[r] = make_float2(mean[i], rstd);
      total[i] = rstd;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      F2 w[4], b[4];
      own.read(weight, n, w);
      own.read(bias, n, b);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = r0 + step * i;
        const bool real = r < a.rows;
        F2 x[4];
        forget_widened(raw[i][n]);
        widen_pairs<kFp32, kVec>(raw[i][n], x);
        if constexpr (kForm && kVec == 8) {
          pack_eight(x, own.lane_of(n), own.lanes, a.groups, real, kForm, a.codes + r * a.groups * kPackGroup,
                     a.scales + r * a.groups);
        } else if constexpr (kForm) {
          F2 p[4];
          to_neighbours(x, turned[threadIdx.x / 32], p);
          uint32_t byte;
          const uint2 c = encode_eight(p, 4, kForm, &byte);
          const int g = turned_group(n, own.lane, own.lanes);
          if (real && g < a.groups) {
            *reinterpret_cast<uint2*>(a.codes + (r * a.groups + g) * kPackGroup + own.lane % 4 * 8) = c;
            if (own.lane % 4 == 0) a.scales[r * a.groups + g] = static_cast<uint8_t>(byte);
          }
        }
        const F2 rstd = both(total[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = fma2(mul2(add2(x[k], less[i]), rstd), w[k], b[k]);
        if (real) {
          store_pairs<kFp32, kVec>(static_cast<char*>(a.out) + (r * a.out_stride + own.at(n)) * kSize, own.lane_of(n),
                                   own.lanes, a.cols - own.at(n), x);
        }
      }
    }
  }
}

template <bool kFp32, int kVec, int kN>
constexpr int kBackwardRows = kN * (kFp32 || kVec == 1 ? 2 : 1) >= 4 ? 1 : 2;

// Rows of whole vectors come through shared memory: a thread's copies of its own
// columns run kStages - 1 turns ahead of it, whatever the barriers of a turn
// make it wait for.  Bytes of a thread's turn:
constexpr int kStages = 2;
template <bool kFp32, int kN, bool kPacked>
constexpr int kTurnBytes = kBackwardRows<kFp32, 8, kN> * kN * (16 * (kFp32 ? 2 : 1) + (kPacked ? 8 : 16 * (kFp32 ? 2 : 1)));

template <bool kFp32, int kVec, int kN, int kForm>
__global__ void __launch_bounds__(kBackwardWarps * 32, 1) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = kBackwardRows<kFp32, kVec, kN>;
  constexpr long long kSize = kFp32 ? 4 : 2;
  constexpr bool kPacked = kForm != 0;  // x comes from its 8-bit form
  constexpr bool kAhead = kVec == 8;
  constexpr int kWords = kFp32 ? 2 : 1;  // 16-byte words of eight elements
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for all of this
  extern __shared__ __align__(16) float tables[];
  __shared__ float buffer[2][kNormWarps][2 * kRows];
  __shared__ __align__(16) float turned[kVec == 1 && kPacked ? kBackwardWarps : 1][256];
  GroupSum<2 * kRows> sum(buffer, a.lanes);
  const Slots<kVec, kN> own{a.lanes, static_cast<int>(threadIdx.x) % a.lanes};
  const int groups = blockDim.x / a.lanes, group = threadIdx.x / a.lanes;
  const long long step = static_cast<long long>(gridDim.x) * groups * kRows;
  const long long mine = blockIdx.x + static_cast<long long>(gridDim.x) * group;
  F2 dw[kN][4] = {}, db[kN][4] = {};
  // the copies' places: [stage][dy's words, then x's or its codes][row][n][thread]
  constexpr int kPitch = kBackwardWarps * 32;
  constexpr int kTurn = kAhead ? kTurnBytes<kFp32, kN, kPacked> * kPitch : 0;
  char* const ring = reinterpret_cast<char*>(tables + kN * 8 * a.lanes);
  auto place = [&](int stage, int i, int n, int word) {
    if (kPacked && word == kWords)
      return ring + stage * kTurn + (kRows * kN * kWords * 16 + (i * kN + n) * 8) * kPitch + threadIdx.x * 8;
    return ring + stage * kTurn + ((kRows * word + i) * kN + n) * 16 * kPitch + threadIdx.x * 16;
  };
  // Where the thread's first words of the next turn to copy lie: moved on where x
  // is whole; beside codes and scales there are no registers for that.
  const long long apart = static_cast<long long>(gridDim.x) * groups;
  const long long x_pitch = a.x_stride * kSize, dy_pitch = a.dy_stride * kSize;
  const char* next_x = static_cast<const char*>(a.x) + mine * x_pitch + own.lane * (16 * kWords);
  const char* next_dy = static_cast<const char*>(a.dy) + mine * dy_pitch + own.lane * (16 * kWords);
  long long next_row = mine;
  auto copy = [&](int stage) {
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = next_row + apart * i;
        if (r >= a.rows) break;
        const char* from = kPacked ? static_cast<const char*>(a.dy) + r * dy_pitch + own.lane * (16 * kWords)
                                   : next_dy + apart * i * dy_pitch;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          if (own.lane_of(n) * 8 >= a.cols) break;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            copy_async<16>(place(stage, i, n, w), from + n * own.lanes * (16 * kWords) + w * 16);
            if constexpr (!kPacked)
              copy_async<16>(place(stage, i, n, kWords + w), next_x + apart * i * x_pitch + n * own.lanes * (16 * kWords) + w * 16);
          }
          if constexpr (kPacked)
            copy_async<8>(place(stage, i, n, kWords), a.codes + r * a.groups * kPackGroup + own.lane_of(n) * 8LL);
        }
      }
      copy_commit();
      next_row += step;
      if constexpr (!kPacked) {
        next_x += step * x_pitch;
        next_dy += step * dy_pitch;
      }
    }
  };
  // what a turn needs beside: the rows' statistics and scales, a turn ahead
  float2 stats[kRows], next_stats[kRows];
  uint32_t scales[kRows][kN], next_scales[kRows][kN];
  auto look_ahead = [&](long long r0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = r0 + static_cast<long long>(gridDim.x) * groups * i;
      next_stats[i] = r < a.rows ? a.stats[r] : make_float2(0.0f, 0.0f);
      if constexpr (kPacked && kAhead) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
          next_scales[i][n] = r < a.rows && own.lane_of(n) * 8 < a.cols ? a.scales[r * a.groups + own.lane_of(n) / 4] : 0u;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy(s);
  look_ahead(mine);
  for (int four = threadIdx.x; four < kN * 2 * a.lanes; four += blockDim.x)
    own.store_four(tables, four, own.load_four(a.weight, a.weight_fp32, four, a.cols, 1.0f));
  __syncthreads();
  int stage = 0;
  for (long long r0 = mine; r0 < a.rows; r0 += step) {
    Eight<kFp32, kVec> raw[kRows][kN], grad[kRows][kN];
    EightCodes codes[kRows][kN];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      stats[i] = next_stats[i];
#pragma unroll
      for (int n = 0; n < kN; ++n) scales[i][n] = kPacked && kAhead ? next_scales[i][n] : 0u;
    }
    look_ahead(r0 + step);
    if constexpr (kAhead) {
      copy((stage + kStages - 1) % kStages);  // where the turn before this one was
      copy_wait<kStages - 1>();
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool real = r0 + static_cast<long long>(gridDim.x) * groups * i < a.rows;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const bool some = real && own.lane_of(n) * 8 < a.cols;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
            if (some) {
              u = *reinterpret_cast<const uint4*>(place(stage, i, n, w));
              if constexpr (!kPacked) v = *reinterpret_cast<const uint4*>(place(stage, i, n, kWords + w));
            }
            grad[i][n].w[4 * w] = u.x; grad[i][n].w[4 * w + 1] = u.y; grad[i][n].w[4 * w + 2] = u.z; grad[i][n].w[4 * w + 3] = u.w;
            raw[i][n].w[4 * w] = v.x; raw[i][n].w[4 * w + 1] = v.y; raw[i][n].w[4 * w + 2] = v.z; raw[i][n].w[4 * w + 3] = v.w;
          }
          if constexpr (kPacked) {
            const uint2 u = some ? *reinterpret_cast<const uint2*>(place(stage, i, n, kWords)) : make_uint2(0u, 0u);
            codes[i][n].w[0] = u.x; codes[i][n].w[1] = u.y; codes[i][n].w[2] = scales[i][n];
          }
        }
      }
      stage = (stage + 1) % kStages;
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = r0 + static_cast<long long>(gridDim.x) * groups * i;
        const bool real = r < a.rows;
        const char* row = static_cast<const char*>(a.x) + r * a.x_stride * kSize;
        const char* drow = static_cast<const char*>(a.dy) + r * a.dy_stride * kSize;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          if constexpr (kPacked) {  // of a group of the warp's, to be turned
            const int g = turned_group(n, own.lane, own.lanes);
            load_codes(a.codes + (r * a.groups + g) * kPackGroup, a.scales + r * a.groups + g, own.lane % 4,
                       real && g < a.groups ? 1 : 0, &codes[i][n]);
          } else {
            load_eight<kFp32, kVec>(row + own.at(n) * kSize, own.lane_of(n), own.lanes, real ? a.cols - own.at(n) : 0,
                                    &raw[i][n]);
          }
          load_eight<kFp32, kVec>(drow + own.at(n) * kSize, own.lane_of(n), own.lanes, real ? a.cols - own.at(n) : 0,
                                  &grad[i][n]);
        }
      }
    }
    // x less the mean, and dy (columns past the last: dy is zero, and what they add to sums, too)
    auto values = [&](int i, int n, F2* d, F2* g) {
      if constexpr (kPacked) {
        widen_codes(codes[i][n], kForm, d);
        if constexpr (kVec == 1) {
          F2 p[4] = {d[0], d[1], d[2], d[3]};
          to_singles(p, turned[threadIdx.x / 32], d);
        }
      } else {
        widen_pairs<kFp32, kVec>(raw[i][n], d);
      }
      widen_pairs<kFp32, kVec>(grad[i][n], g);
      const F2 less = both(-stats[i].x);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = add2(d[k], less);
    };
    F2 one[kRows] = {}, two[kRows] = {};
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      F2 w[4];
      own.read(tables, n, w);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        F2 xn[4], g[4];
        values(i, n, xn, g);
        const F2 rstd = both(stats[i].y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xn[k] = mul2(xn[k], rstd);
          dw[n][k] = fma2(g[k], xn[k], dw[n][k]);
          db[n][k] = add2(db[n][k], g[k]);
          g[k] = mul2(g[k], w[k]);
          one[i] = add2(one[i], g[k]);
          two[i] = fma2(g[k], xn[k], two[i]);
        }
      }
    }
    float total[2 * kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      total[2 * i] = sum_of(one[i]);
      total[2 * i + 1] = sum_of(two[i]);
    }
    sum(total);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      F2 w[4];
      own.read(tables, n, w);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long r = r0 + static_cast<long long>(gridDim.x) * groups * i;
        if (r >= a.rows) continue;
        const F2 m1 = both(a.center ? -total[2 * i] * a.inv_cols : 0.0f), rstd = both(stats[i].y);
        const F2 m2 = both(-total[2 * i + 1] * a.inv_cols * stats[i].y);  // of x less the mean
        F2 d[4], g[4];
        if constexpr (kPacked) forget_widened(codes[i][n]);
        else forget_widened(raw[i][n]);
        forget_widened(grad[i][n]);
        values(i, n, d, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] = mul2(rstd, fma2(d[k], m2, fma2(g[k], w[k], m1)));
        store_pairs<kFp32, kVec>(static_cast<char*>(a.out) + (r * a.out_stride + own.at(n)) * kSize, own.lane_of(n),
                                 own.lanes, a.cols - own.at(n), g);
      }
    }
  }
  if constexpr (kAhead) copy_wait<0>();
  if (!a.partials) return;
  // the CTA's sums: one group after another adds its own, in the weights' place
  float* part = a.partials + static_cast<long long>(blockIdx.x) * 2 * a.cols;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which && !a.want_bias) break;
    for (int turn = 0; turn < groups; ++turn) {
      __syncthreads();
      if (turn != group) continue;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float mine[8];
        from_pairs(which ? db[n] : dw[n], mine);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = own.slot(own.column_of(n, k));
          const float s = mine[k];
          tables[at] = turn ? tables[at] + s : s;
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) part[which * a.cols + c] = tables[own.slot(c)];
    __syncthreads();
  }
}

// ---- rows that no CTA holds: any number of columns, any alignment --------------
__device__ __forceinline__ float cta_sum(float v, float* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kWideThreads / 32; ++w) v += shared[w];
  return v;
}

template <bool kFp32>
__device__ __forceinline__ float element(const void* p, long long at) {
  return load_scalar(p, kFp32, at);
}
// Element c of a row of 8-bit codes.
__device__ __forceinline__ float kept(const NormArgs& a, long long row, int c) {
  return decode1(a.codes[row * a.groups * kPackGroup + c], a.form) * scale_value(a.scales[row * a.groups + c / kPackGroup]);
}

template <bool kFp32>
__global__ void __launch_bounds__(kWideThreads) norm_wide_forward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[kWideThreads / 32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const long long at = r * a.x_stride;
    float mean = 0.0f, total = 0.0f;
    if (a.center) {
      for (int c = threadIdx.x; c < a.cols; c += kWideThreads) mean += element<kFp32>(a.x, at + c);
      mean = cta_sum(mean, shared) * a.inv_cols;
    }
    for (int c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float d = element<kFp32>(a.x, at + c) - mean;
      total = fmaf(d, d, total);
    }
    const float rstd = rsqrtf(fmaf(cta_sum(total, shared), a.inv_cols, a.eps));
    if (a.stats && threadIdx.x == 0) a.stats[r] = make_float2(mean, rstd);
    // a warp's 32 columns are a group
    for (int c0 = threadIdx.x & ~31; c0 < a.cols; c0 += kWideThreads) {
      const int c = c0 + threadIdx.x % 32;
      const float x = c < a.cols ? element<kFp32>(a.x, at + c) : 0.0f;
      if (a.form != 0) {
        const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu), a.form);
        const uint32_t code = byte == 255u ? 0u : encode1(x * inverse_scale(byte), a.form);
        a.codes[r * a.groups * kPackGroup + c] = static_cast<uint8_t>(code);
        if (threadIdx.x % 32 == 0) a.scales[r * a.groups + c0 / kPackGroup] = static_cast<uint8_t>(byte);
      }
      if (c < a.cols) {
        const float w = a.weight ? load_scalar(a.weight, a.weight_fp32, c) : 1.0f;
        const float b = a.bias ? load_scalar(a.bias, a.weight_fp32, c) : 0.0f;
        store_scalar(a.out, kFp32, r * a.out_stride + c, fmaf((x - mean) * rstd, w, b));
      }
    }
  }
}

template <bool kFp32, bool kPacked>
__device__ __forceinline__ float normed(const NormArgs& a, long long r, int c, float2 stats) {
  const float x = kPacked ? kept(a, r, c) : element<kFp32>(a.x, r * a.x_stride + c);
  return (x - stats.x) * stats.y;
}

// Sums of a share of the rows for kWideThreads columns (before the rows' pass,
// which may write dx over x or dy).
template <bool kFp32, bool kPacked>
__global__ void __launch_bounds__(kWideThreads) norm_wide_columns_kernel(const __grid_constant__ NormArgs a) {
  const long long c = static_cast<long long>(blockIdx.x) * kWideThreads + threadIdx.x;
  if (c >= a.cols) return;
  const long long share = (a.rows + a.parts - 1) / a.parts, begin = blockIdx.y * share;
  const long long end = begin + share < a.rows ? begin + share : a.rows;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (long long r = begin; r < end; ++r) {
    const float g = element<kFp32>(a.dy, r * a.dy_stride + c);
    dw = fmaf(g, normed<kFp32, kPacked>(a, r, static_cast<int>(c), a.stats[r]), dw);
    db += g;
  }
  float* part = a.partials + static_cast<long long>(blockIdx.y) * 2 * a.cols;
  part[c] = dw;
  part[a.cols + c] = db;
}

template <bool kFp32, bool kPacked>
__global__ void __launch_bounds__(kWideThreads) norm_wide_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[kWideThreads / 32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float2 stats = a.stats[r];
    float m1 = 0.0f, m2 = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float g = element<kFp32>(a.dy, r * a.dy_stride + c) * (a.weight ? load_scalar(a.weight, a.weight_fp32, c) : 1.0f);
      m1 += g;
      m2 = fmaf(g, normed<kFp32, kPacked>(a, r, c, stats), m2);
    }
    m1 = a.center ? cta_sum(m1, shared) * a.inv_cols : 0.0f;
    m2 = cta_sum(m2, shared) * a.inv_cols;
    for (int c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float g = element<kFp32>(a.dy, r * a.dy_stride + c) * (a.weight ? load_scalar(a.weight, a.weight_fp32, c) : 1.0f);
      const float xn = normed<kFp32, kPacked>(a, r, c, stats);
      store_scalar(a.out, kFp32, r * a.out_stride + c, stats.y * fmaf(-xn, m2, g - m1));
    }
  }
}

// The gradients of weight and bias from the parts' sums: 32 columns per CTA,
// every warp a contiguous share of the parts, then warp after warp.
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float sums[kJoinWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, which = blockIdx.y;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  const int share = (a.parts + kJoinWarps - 1) / kJoinWarps, begin = warp * share;
  const int end = begin + share < a.parts ? begin + share : a.parts;
  float s = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < a.cols) {
#pragma unroll 8
    for (int p = begin; p < end; ++p) s += a.partials[(static_cast<long long>(p) * 2 + which) * a.cols + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int v = 0; v < kJoinWarps; ++v) s += sums[v][lane];
  void* to = which ? a.dbias : a.dweight;
  if (to) store_scalar(to, a.dgrad_fp32, c, s);
}

// ---- host ----------------------------------------------------------------------
// How a row is held: by `lanes` lanes of a warp (up to 16), by a group of `lanes`
// threads of a CTA of `threads`, kN times eight columns each, or (0) by none.
struct Shape {
  int lanes, threads, n;
  bool vec;
};
// most: the largest kN that the pass has registers for (single elements: 2).
// Where every row can have an SM to itself, it is spread over as many warps as
// there are (1 row of 2048: 2.6 us of device time, 3.7 us as one warp of many).
Shape shape_of(int cols, long long rows, bool vec, int most, int cta_warps) {
  if (cols > kNormWidest) return {0, kWideThreads, 0, false};
  const int eights = (cols + 7) / 8;
  if (vec && cols <= kLaneCols) return {power_of_two(eights), kLaneThreads, 1, true};
  if (!vec && most > 2) most = 2;
  const bool alone = rows <= sm_count();
  const int warps = (eights + 31) / 32;
  int n = 1;
  while (n < most && (alone ? n * cta_warps < warps : n < warps)) n *= 2;
  const int lanes = (warps + n - 1) / n * 32, groups = alone ? 1 : cta_warps * 32 / lanes;
  return {lanes, groups * lanes, n, vec};
}
Shape forward_shape(int cols, long long rows, bool vec, bool fp32) {
  return shape_of(cols, rows, vec, fp32 ? 4 : 8, kForwardWarps);
}
Shape backward_shape(int cols, long long rows, bool vec) { return shape_of(cols, rows, vec, 2, kBackwardWarps); }

// CTAs for all rows: what is resident at once, at most.
int norm_ctas(const Shape& s, long long rows) {
  const bool small = s.lanes > 0 && s.lanes < 32;
  const long long per_cta = small ? s.threads / s.lanes : 1;
  const long long want = (rows + per_cta - 1) / per_cta, per_sm = s.lanes == 0 ? 2048 / kWideThreads : small ? kLaneCtas : 1;
  const long long most = per_sm * sm_count();
  return static_cast<int>(want < most ? want : most);
}
// Parts of the rows whose column sums are joined.
int wide_parts(long long rows) { return static_cast<int>(rows < 32 ? (rows ? rows : 1) : 32); }
int parts_of(const Shape& s, long long rows) { return s.lanes ? norm_ctas(s, rows) : wide_parts(rows); }
// ... whether or not the tensors turn out to be aligned, for the workspace.
int most_parts(int cols, long long rows) {
  const int a = parts_of(backward_shape(cols, rows, false), rows), b = parts_of(backward_shape(cols, rows, true), rows);
  return a > b ? a : b;
}

// kMost: of dynamic shared memory.
template <auto kKernel, int kMost>
void launch_with(const NormArgs& a, const Shape& s, int ctas, int bytes, cudaStream_t st) {
  if (bytes > 20 * 1024 && allow_shared<kKernel, kMost>() != cudaSuccess) return;  // reported as the launch's error
  kKernel<<<ctas, s.threads, bytes, st>>>(a);
}

template <bool kFp32, int kVec, int kN>
void launch_forward_n(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  const int bytes = 2 * kN * 8 * s.lanes * static_cast<int>(sizeof(float));
  if (a.form == 0) launch_with<norm_forward_kernel<kFp32, kVec, kN, 0>, 64 * 1024>(a, s, ctas, bytes, st);
  else if (a.form == kPackE4m3) launch_with<norm_forward_kernel<kFp32, kVec, kN, kPackE4m3>, 64 * 1024>(a, s, ctas, bytes, st);
  else launch_with<norm_forward_kernel<kFp32, kVec, kN, kPackInt8>, 64 * 1024>(a, s, ctas, bytes, st);
}
template <bool kFp32, int kVec>
void launch_forward(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  if constexpr (kVec == 8) {
    if (s.lanes < 32) return norm_lanes_forward_kernel<kFp32><<<ctas, s.threads, 0, st>>>(a);
    if (s.n == 4) return launch_forward_n<kFp32, kVec, 4>(a, s, ctas, st);
    if constexpr (!kFp32) {
      if (s.n == 8) return launch_forward_n<kFp32, kVec, 8>(a, s, ctas, st);
    }
  }
  if (s.n == 2) launch_forward_n<kFp32, kVec, 2>(a, s, ctas, st);
  else launch_forward_n<kFp32, kVec, 1>(a, s, ctas, st);
}
template <bool kFp32, int kVec, int kN, int kForm>
void launch_backward_n(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  const int bytes = kN * 8 * s.lanes * static_cast<int>(sizeof(float)) +
                    (kVec == 8 ? kStages * kTurnBytes<kFp32, kN, kForm != 0> * kBackwardWarps * 32 : 0);
  launch_with<norm_backward_kernel<kFp32, kVec, kN, kForm>, (kVec == 8 ? 225 : 32) * 1024>(a, s, ctas, bytes, st);
}
template <bool kFp32, int kVec, int kForm>
void launch_backward_form(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  if constexpr (kVec == 8) {
    if (s.lanes < 32) return norm_lanes_backward_kernel<kFp32, kForm != 0><<<ctas, s.threads, 0, st>>>(a);
  }
  if (s.n == 2) launch_backward_n<kFp32, kVec, 2, kForm>(a, s, ctas, st);
  else launch_backward_n<kFp32, kVec, 1, kForm>(a, s, ctas, st);
}
template <bool kFp32, int kVec>
void launch_backward(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  if (a.form == 0) launch_backward_form<kFp32, kVec, 0>(a, s, ctas, st);
  else if (a.form == kPackE4m3) launch_backward_form<kFp32, kVec, kPackE4m3>(a, s, ctas, st);
  else launch_backward_form<kFp32, kVec, kPackInt8>(a, s, ctas, st);
}
template <bool kFp32, bool kPacked>
void launch_wide_backward(const NormArgs& a, int ctas, cudaStream_t st) {
  if (a.partials) {
    const dim3 grid((a.cols + kWideThreads - 1) / kWideThreads, a.parts);
    norm_wide_columns_kernel<kFp32, kPacked><<<grid, kWideThreads, 0, st>>>(a);
  }
  norm_wide_backward_kernel<kFp32, kPacked><<<ctas, kWideThreads, 0, st>>>(a);
}

zero_status check_norm(const zero_norm_config* c, int64_t rows) {
  if (!c) return refuse(ZERO_EINVAL, "config is NULL");
  if (rows < 0) return refuse(ZERO_EINVAL, "rows is negative");
  if (c->cols < 1 || c->cols > (1 << 24)) return refuse(ZERO_EINVAL, "cols not in 1..2^24");
  if (!is_dtype(c->dtype) || !is_dtype(c->weight_dtype))
    return refuse(ZERO_EINVAL, "a dtype is neither bf16 (0) nor fp32 (1)");
  if (c->center != 0 && c->center != 1) return refuse(ZERO_EINVAL, "center must be 0 or 1");
  if (!(c->eps >= 0.0f) || !std::isfinite(c->eps)) return refuse(ZERO_EINVAL, "eps must be finite and >= 0");
  return ZERO_OK;
}

zero_status check_packed(const zero_packed* p, NormArgs* a) {
  if (p->format != ZERO_PACK_E4M3 && p->format != ZERO_PACK_INT8)
    return refuse(ZERO_EINVAL, "the 8-bit format is neither e4m3 (0) nor int8 (1)");
  if (misplaced(p->codes, 16) || !p->scales) return refuse(ZERO_EINVAL, "codes or scales are NULL or misaligned");
  a->form = p->format == ZERO_PACK_E4M3 ? kPackE4m3 : kPackInt8;
  a->codes = static_cast<uint8_t*>(p->codes);
  a->scales = static_cast<uint8_t*>(p->scales);
  return ZERO_OK;
}

zero_status check_matrix(const void* p, int64_t stride, int dtype, const char* text) {
  if (misplaced(p, dtype_bytes(dtype)) || stride < 0) return refuse(ZERO_EINVAL, text);
  return ZERO_OK;
}

void fill(const zero_norm_config* c, int64_t rows, NormArgs* a) {
  a->rows = rows;
  a->cols = static_cast<int>(c->cols);
  a->inv_cols = static_cast<float>(1.0 / static_cast<double>(c->cols));
  a->eps = c->eps;
  a->weight_fp32 = c->weight_dtype == ZERO_GRAD_FP32;
  a->center = c->center;
  a->groups = (a->cols + kPackGroup - 1) / kPackGroup;
}

}  // namespace

}  // namespace zfs

extern "C" {

zero_status zero_layer_norm(const zero_norm_config* cfg, int64_t rows, const void* x, int64_t x_stride,
                            const void* weight, const void* bias, void* y, int64_t y_stride, float* stats,
                            const zero_packed* packed, void* stream) {
  using namespace zfs;
  zero_status st = check_norm(cfg, rows);
  if (st != ZERO_OK) return st;
  if (rows == 0) return ZERO_OK;
  NormArgs a{};
  fill(cfg, rows, &a);
  const int vsz = dtype_bytes(cfg->weight_dtype);
  if ((st = check_matrix(x, x_stride, cfg->dtype, "x is NULL or misaligned, or its stride negative")) != ZERO_OK) return st;
  if ((st = check_matrix(y, y_stride, cfg->dtype, "y is NULL or misaligned, or its stride negative")) != ZERO_OK) return st;
  if (rows_overlap(y_stride, rows, cfg->cols)) return refuse(ZERO_EINVAL, "y's stride makes its rows overlap");
  if ((weight && misplaced(weight, vsz)) || (bias && misplaced(bias, vsz)))
    return refuse(ZERO_EINVAL, "weight or bias is misaligned");
  if (stats && misplaced(stats, 8)) return refuse(ZERO_EINVAL, "stats is misaligned");
  if (packed && (st = check_packed(packed, &a)) != ZERO_OK) return st;
  a.x = x;
  a.x_stride = x_stride;
  a.out = y;
  a.out_stride = y_stride;
  a.weight = weight;
  a.bias = bias;
  a.stats = reinterpret_cast<float2*>(stats);
  const bool vec = a.cols % 8 == 0 && rows_aligned(x, x_stride, rows, cfg->dtype) && rows_aligned(y, y_stride, rows, cfg->dtype);
  const bool fp32 = cfg->dtype == ZERO_GRAD_FP32;
  const Shape s = forward_shape(a.cols, rows, vec, fp32);
  const int ctas = norm_ctas(s, rows);
  a.lanes = s.lanes;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.lanes == 0) {
    if (fp32) norm_wide_forward_kernel<true><<<ctas, kWideThreads, 0, cs>>>(a);
    else norm_wide_forward_kernel<false><<<ctas, kWideThreads, 0, cs>>>(a);
  } else if (s.vec) {
    if (fp32) launch_forward<true, 8>(a, s, ctas, cs);
    else launch_forward<false, 8>(a, s, ctas, cs);
  } else {
    if (fp32) launch_forward<true, 1>(a, s, ctas, cs);
    else launch_forward<false, 1>(a, s, ctas, cs);
  }
  return launch_status("layer norm launch");
}

zero_status zero_layer_norm_backward_workspace_bytes(const zero_norm_config* cfg, int64_t rows, int64_t* bytes) {
  if (!bytes) return zfs::refuse(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_norm(cfg, rows);
  if (st != ZERO_OK) return st;
  *bytes = static_cast<int64_t>(zfs::most_parts(static_cast<int>(cfg->cols), rows)) * 2 * cfg->cols * 4;
  return ZERO_OK;
}

zero_status zero_layer_norm_backward(const zero_norm_config* cfg, int64_t rows, const void* dy, int64_t dy_stride,
                                     const void* x, int64_t x_stride, const zero_packed* packed, const void* weight,
                                     const float* stats, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                     int32_t dgrad_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  using namespace zfs;
  zero_status st = check_norm(cfg, rows);
  if (st != ZERO_OK) return st;
  if (!is_dtype(dgrad_dtype)) return refuse(ZERO_EINVAL, "dgrad_dtype is neither bf16 (0) nor fp32 (1)");
  const int dsz = dtype_bytes(dgrad_dtype);
  if ((dweight && misplaced(dweight, dsz)) || (dbias && misplaced(dbias, dsz)))
    return refuse(ZERO_EINVAL, "a gradient of weight or bias is misaligned");
  NormArgs a{};
  fill(cfg, rows, &a);
  a.dweight = dweight;
  a.dbias = dbias;
  a.dgrad_fp32 = dgrad_dtype == ZERO_GRAD_FP32;
  a.want_bias = dbias != nullptr;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    if ((st = check_matrix(dy, dy_stride, cfg->dtype, "dy is NULL or misaligned, or its stride negative")) != ZERO_OK) return st;
    if ((st = check_matrix(dx, dx_stride, cfg->dtype, "dx is NULL or misaligned, or its stride negative")) != ZERO_OK) return st;
    if (rows_overlap(dx_stride, rows, cfg->cols)) return refuse(ZERO_EINVAL, "dx's stride makes its rows overlap");
    if (packed) {
      if ((st = check_packed(packed, &a)) != ZERO_OK) return st;
    } else if ((st = check_matrix(x, x_stride, cfg->dtype, "x is NULL or misaligned, or its stride negative")) != ZERO_OK) {
      return st;
    }
    if (weight && misplaced(weight, dtype_bytes(cfg->weight_dtype))) return refuse(ZERO_EINVAL, "weight is misaligned");
    if (misplaced(stats, 8)) return refuse(ZERO_EINVAL, "stats is NULL or misaligned");
    if (dweight || dbias) {
      int64_t need = 0;
      zero_layer_norm_backward_workspace_bytes(cfg, rows, &need);
      if (misplaced(workspace, 16)) return refuse(ZERO_EINVAL, "workspace is NULL or not 16-byte aligned");
      if (workspace_bytes < need) return refuse(ZERO_EINVAL, "workspace is too small");
      a.partials = static_cast<float*>(workspace);
    }
    a.x = x;
    a.x_stride = x_stride;
    a.dy = dy;
    a.dy_stride = dy_stride;
    a.out = dx;
    a.out_stride = dx_stride;
    a.weight = weight;
    a.stats = const_cast<float2*>(reinterpret_cast<const float2*>(stats));
    const bool vec = a.cols % 8 == 0 && (packed || rows_aligned(x, x_stride, rows, cfg->dtype)) &&
                     rows_aligned(dy, dy_stride, rows, cfg->dtype) && rows_aligned(dx, dx_stride, rows, cfg->dtype);
    const Shape s = backward_shape(a.cols, rows, vec);
    const int ctas = norm_ctas(s, rows);
    a.lanes = s.lanes;
    a.parts = parts_of(s, rows);
    const bool fp32 = cfg->dtype == ZERO_GRAD_FP32;
    if (s.lanes == 0) {
      if (fp32) packed ? launch_wide_backward<true, true>(a, ctas, cs) : launch_wide_backward<true, false>(a, ctas, cs);
      else packed ? launch_wide_backward<false, true>(a, ctas, cs) : launch_wide_backward<false, false>(a, ctas, cs);
    } else if (s.vec) {
      if (fp32) launch_backward<true, 8>(a, s, ctas, cs);
      else launch_backward<false, 8>(a, s, ctas, cs);
    } else {
      if (fp32) launch_backward<true, 1>(a, s, ctas, cs);
      else launch_backward<false, 1>(a, s, ctas, cs);
    }
    if ((st = launch_status("layer norm backward launch")) != ZERO_OK) return st;
  }
  if (!dweight && !dbias) return ZERO_OK;
  launch_after(norm_join_kernel, dim3((a.cols + 31) / 32, dbias ? 2 : 1), dim3(kJoinThreads), 0, cs, a);
  return launch_status("layer norm weight gradient launch");
}

}  // extern "C"
