// Layer norm over the columns of a matrix, forward and backward, with the
// input's 8-bit form written and read in the same passes, and its C calls.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd weight + bias
// (mean 0 without centring).  Backward, with xn = (x - mean) rstd, g = dy weight:
//   dx = rstd (g - sum g / n - xn sum (g xn) / n),  dweight = sum dy xn,
//   dbias = sum dy
// (without the sum of g alone where nothing was centred).

#include <cmath>

#include "zero_flatstep.h"
#include "zero_norm_internal.h"
#include "zero_rows.cuh"
#include "zero_rows_host.h"

namespace zfs {
namespace {

constexpr int kNormThreads = 256;   // threads of a CTA that holds several rows
constexpr int kNormWidest = 8192;   // columns that a CTA of 1024 threads holds
constexpr int kWideThreads = 512;   // threads of a CTA that walks over a row

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

// Sums of kN values over the lanes that hold a row: by shuffles within a group
// of lanes of a warp, or over the CTA through `shared` (two alternating
// buffers, so that one barrier a sum is enough).
template <bool kLanes, int kN>
struct RowSum {
  float (*buffer)[32][kN];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[kN], int lanes) {
    const int width = kLanes ? lanes : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o < width) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
    }
    if constexpr (!kLanes) {
      if (threadIdx.x % 32 == 0) {
#pragma unroll
        for (int i = 0; i < kN; ++i) buffer[turn][threadIdx.x / 32][i] = v[i];
      }
      __syncthreads();
      const int warps = lanes / 32;
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = 0.0f;
      for (int w = 0; w < warps; ++w) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += buffer[turn][w][i];
      }
      turn ^= 1;
    }
  }
};

template <int kVec>
__device__ __forceinline__ void load_vector(const void* p, bool fp32, int lane, int lanes, int cols, float other, float* w) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = column<kVec>(k, lane, lanes);
    w[k] = p && c < cols ? load_scalar(p, fp32, c) : other;
  }
}

// kLanes: a.lanes lanes of a warp hold a row, else the CTA does.
template <bool kFp32, int kVec, bool kLanes, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = 2;  // in flight
  constexpr long long kSize = kFp32 ? 4 : 2;
  __shared__ float buffer[2][32][kRows];
  RowSum<kLanes, kRows> sum{buffer};
  const int lanes = a.lanes, lane = kLanes ? threadIdx.x % lanes : threadIdx.x;
  const int per_cta = kLanes ? kThreads / lanes : 1;
  float w[8], b[8];
  load_vector<kVec>(a.weight, a.weight_fp32, lane, lanes, a.cols, 1.0f, w);
  load_vector<kVec>(a.bias, a.weight_fp32, lane, lanes, a.cols, 0.0f, b);
  const long long step = static_cast<long long>(gridDim.x) * per_cta;
  const long long mine = static_cast<long long>(blockIdx.x) * per_cta + (kLanes ? threadIdx.x / lanes : 0);
  // all threads take the same number of turns
  for (long long r0 = 0; static_cast<long long>(blockIdx.x) * per_cta + r0 < a.rows; r0 += step * kRows) {
    Eight<kFp32, kVec> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + r0 + step * i;
      load_eight<kFp32, kVec>(static_cast<const char*>(a.x) + r * a.x_stride * kSize, lane, lanes,
                              r < a.rows ? a.cols : 0, &raw[i]);
    }
    float x[kRows][8], mean[kRows], total[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      widen_eight<kFp32, kVec>(raw[i], x[i]);
      mean[i] = 0.0f;
    }
    if (a.center) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mean[i] += x[i][k];
      }
      sum(mean, lanes);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      mean[i] *= a.inv_cols;
      total[i] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = column<kVec>(k, lane, lanes) < a.cols ? x[i][k] - mean[i] : 0.0f;
        total[i] = fmaf(d, d, total[i]);
      }
    }
    sum(total, lanes);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + r0 + step * i;
      const bool real = r < a.rows;
      if (a.form != 0) {
        pack_eight<kVec>(x[i], lane, lanes, a.groups, real, a.form, a.codes + r * a.groups * kPackGroup,
                         a.scales + r * a.groups);
      }
      const float rstd = rsqrtf(fmaf(total[i], a.inv_cols, a.eps));
      if (a.stats && real && lane == 0) a.stats[r] = make_float2(mean[i], rstd);
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = fmaf((x[i][k] - mean[i]) * rstd, w[k], b[k]);
      if (real) {
        store_eight<kFp32, kVec>(static_cast<char*>(a.out) + r * a.out_stride * kSize, lane, lanes, a.cols, y);
      }
    }
  }
}

// kPacked: x comes from its 8-bit form.
template <bool kFp32, int kVec, bool kLanes, int kThreads, bool kPacked>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = kThreads > 256 ? 1 : 2;
  constexpr long long kSize = kFp32 ? 4 : 2;
  __shared__ float buffer[2][32][2 * kRows];
  RowSum<kLanes, 2 * kRows> sum{buffer};
  const int lanes = a.lanes, lane = kLanes ? threadIdx.x % lanes : threadIdx.x;
  const int per_cta = kLanes ? kThreads / lanes : 1;
  float w[8], dw[8] = {}, db[8] = {};
  load_vector<kVec>(a.weight, a.weight_fp32, lane, lanes, a.cols, 1.0f, w);
  const long long step = static_cast<long long>(gridDim.x) * per_cta;
  const long long mine = static_cast<long long>(blockIdx.x) * per_cta + (kLanes ? threadIdx.x / lanes : 0);
  for (long long r0 = 0; static_cast<long long>(blockIdx.x) * per_cta + r0 < a.rows; r0 += step * kRows) {
    Eight<kFp32, kVec> raw[kRows], grad[kRows];
    EightCodes<kVec> codes[kRows];
    float2 stats[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + r0 + step * i;
      const bool real = r < a.rows;
      stats[i] = real ? a.stats[r] : make_float2(0.0f, 0.0f);
      if constexpr (kPacked) {
        load_codes<kVec>(a.codes + r * a.groups * kPackGroup, a.scales + r * a.groups, lane, lanes,
                         real ? a.groups : 0, &codes[i]);
      } else {
        load_eight<kFp32, kVec>(static_cast<const char*>(a.x) + r * a.x_stride * kSize, lane, lanes,
                                real ? a.cols : 0, &raw[i]);
      }
      load_eight<kFp32, kVec>(static_cast<const char*>(a.dy) + r * a.dy_stride * kSize, lane, lanes,
                              real ? a.cols : 0, &grad[i]);
    }
    float xn[kRows][8], g[kRows][8], total[2 * kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kPacked) widen_codes<kVec>(codes[i], a.form, xn[i]);
      else widen_eight<kFp32, kVec>(raw[i], xn[i]);
      widen_eight<kFp32, kVec>(grad[i], g[i]);
      total[2 * i] = total[2 * i + 1] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // columns past the last: nothing of the mean, of the row's inf or NaN
        xn[i][k] = column<kVec>(k, lane, lanes) < a.cols ? (xn[i][k] - stats[i].x) * stats[i].y : 0.0f;
        dw[k] = fmaf(g[i][k], xn[i][k], dw[k]);
        db[k] += g[i][k];
        g[i][k] *= w[k];
        total[2 * i] += g[i][k];
        total[2 * i + 1] = fmaf(g[i][k], xn[i][k], total[2 * i + 1]);
      }
    }
    sum(total, lanes);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long r = mine + r0 + step * i;
      if (r >= a.rows) continue;
      const float m1 = a.center ? total[2 * i] * a.inv_cols : 0.0f, m2 = total[2 * i + 1] * a.inv_cols;
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = stats[i].y * fmaf(-xn[i][k], m2, g[i][k] - m1);
      store_eight<kFp32, kVec>(static_cast<char*>(a.out) + r * a.out_stride * kSize, lane, lanes, a.cols, d);
    }
  }
  if (!a.partials) return;
  float* part = a.partials + static_cast<long long>(blockIdx.x) * 2 * a.cols;
  if constexpr (kLanes) {
    // over the groups of a warp, then over the warps
    __shared__ float sums[2][kThreads / 32][256];
    const int warp = threadIdx.x / 32;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      for (int o = lanes; o < 32; o <<= 1) {
        dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
        db[k] += __shfl_xor_sync(0xffffffffu, db[k], o);
      }
      if (threadIdx.x % 32 < lanes) {
        sums[0][warp][column<kVec>(k, lane, lanes)] = dw[k];
        sums[1][warp][column<kVec>(k, lane, lanes)] = db[k];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float s = 0.0f;
        for (int v = 0; v < kThreads / 32; ++v) s += sums[which][v][c];
        part[which * a.cols + c] = s;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column<kVec>(k, lane, lanes);
      if (c < a.cols) {
        part[c] = dw[k];
        if (a.want_bias) part[a.cols + c] = db[k];
      }
    }
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
// How a row is held: by `lanes` lanes of a warp, by a CTA of `lanes` threads, or
// (0) by none.
struct Shape {
  int lanes, threads;
  bool vec;
};
Shape shape_of(int cols, bool vec) {
  if (cols > kNormWidest) return {0, kWideThreads, false};
  const int need = vec ? cols / 8 : (cols + 7) / 8;
  if (need <= 32) return {vec ? power_of_two(need) : 32, kNormThreads, vec};
  const int threads = (need + 31) / 32 * 32;
  return {threads, threads, vec};
}

// CTAs for all rows, at most 2048 threads an SM.
int norm_ctas(const Shape& s, long long rows) {
  const long long per_cta = s.lanes && s.lanes <= 32 ? s.threads / s.lanes : 1;
  const long long want = (rows + per_cta - 1) / per_cta, most = static_cast<long long>(sm_count()) * (2048 / s.threads);
  return static_cast<int>(want < most ? want : most);
}
// Parts of the rows whose column sums are joined; the same whether or not the
// tensors turn out to be aligned, for the workspace.
int wide_parts(long long rows) { return static_cast<int>(rows < 32 ? (rows ? rows : 1) : 32); }
int most_parts(int cols, long long rows) {
  if (cols > kNormWidest) return wide_parts(rows);
  const int a = norm_ctas(shape_of(cols, false), rows);
  const int b = cols % 8 ? a : norm_ctas(shape_of(cols, true), rows);
  return a > b ? a : b;
}

template <bool kFp32, int kVec>
void launch_forward(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  if (s.lanes <= 32) norm_forward_kernel<kFp32, kVec, true, kNormThreads><<<ctas, s.threads, 0, st>>>(a);
  else if (s.threads <= 256) norm_forward_kernel<kFp32, kVec, false, 256><<<ctas, s.threads, 0, st>>>(a);
  else norm_forward_kernel<kFp32, kVec, false, 1024><<<ctas, s.threads, 0, st>>>(a);
}
template <bool kFp32, int kVec, bool kPacked>
void launch_backward(const NormArgs& a, const Shape& s, int ctas, cudaStream_t st) {
  if (s.lanes <= 32) norm_backward_kernel<kFp32, kVec, true, kNormThreads, kPacked><<<ctas, s.threads, 0, st>>>(a);
  else if (s.threads <= 256) norm_backward_kernel<kFp32, kVec, false, 256, kPacked><<<ctas, s.threads, 0, st>>>(a);
  else norm_backward_kernel<kFp32, kVec, false, 1024, kPacked><<<ctas, s.threads, 0, st>>>(a);
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

unsigned int norm_debug_failures() {
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
  const Shape s = shape_of(a.cols, vec);
  const int ctas = norm_ctas(s, rows);
  a.lanes = s.lanes;
  const bool fp32 = cfg->dtype == ZERO_GRAD_FP32;
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
    const Shape s = shape_of(a.cols, vec);
    const int ctas = norm_ctas(s, rows);
    a.lanes = s.lanes;
    a.parts = s.lanes ? ctas : wide_parts(rows);
    const bool fp32 = cfg->dtype == ZERO_GRAD_FP32;
    if (s.lanes == 0) {
      if (fp32) packed ? launch_wide_backward<true, true>(a, ctas, cs) : launch_wide_backward<true, false>(a, ctas, cs);
      else packed ? launch_wide_backward<false, true>(a, ctas, cs) : launch_wide_backward<false, false>(a, ctas, cs);
    } else if (s.vec) {
      if (fp32) packed ? launch_backward<true, 8, true>(a, s, ctas, cs) : launch_backward<true, 8, false>(a, s, ctas, cs);
      else packed ? launch_backward<false, 8, true>(a, s, ctas, cs) : launch_backward<false, 8, false>(a, s, ctas, cs);
    } else {
      if (fp32) packed ? launch_backward<true, 1, true>(a, s, ctas, cs) : launch_backward<true, 1, false>(a, s, ctas, cs);
      else packed ? launch_backward<false, 1, true>(a, s, ctas, cs) : launch_backward<false, 1, false>(a, s, ctas, cs);
    }
    if ((st = launch_status("layer norm backward launch")) != ZERO_OK) return st;
  }
  if (!dweight && !dbias) return ZERO_OK;
  launch_after(norm_join_kernel, dim3((a.cols + 31) / 32, dbias ? 2 : 1), dim3(kJoinThreads), 0, cs, a);
  return launch_status("layer norm weight gradient launch");
}

}  // extern "C"
