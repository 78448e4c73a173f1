// Norm of the queries and keys of every head with the position rotation in
// the same pass, forward and backward, and their C calls.
//
//   y = x * rstd * gain,  rstd = 1 / sqrt(mean(x^2) + eps)
//   out = R(position) y   (R turns pairs of the first rotary_dim elements)
// backward, with xn = x * rstd and h = R^T dout:
//   dx = rstd * (gain h - xn * mean(gain h xn)),  dgain = sum h xn
//
// A head is read once and written once; everything between is fp32 in
// registers and shared memory.  One warp per head of a token.

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

// The gain gradients from the CTAs' sums, in CTA order.
__global__ void __launch_bounds__(kQkThreads) qk_gain_kernel(const __grid_constant__ QkArgs a, int ctas) {
  const int d = blockIdx.x * kQkThreads + threadIdx.x;
  if (d >= 2 * a.dim) return;
  const int which = d / a.dim;
  if (!a.dgain[which]) return;
  double s = 0.0;
  for (int c = 0; c < ctas; ++c) s += a.partials[static_cast<long long>(c) * 2 * a.dim + d];
  if (a.dgain_fp32) store_one<true>(a.dgain[which], d % a.dim, static_cast<float>(s));
  else store_one<false>(a.dgain[which], d % a.dim, static_cast<float>(s));
}

int qk_ctas(long long rows) {
  const long long want = (rows + kQkWarps - 1) / kQkWarps, most = 4LL * sm_count();
  return static_cast<int>(want < 1 ? 0 : want < most ? want : most);
}

zero_status report(zero_status st, const char* text) {
  zfs_report_error(nullptr, st, text);
  return st;
}

bool bad(const void* p, int esz, int device) {
  if (!p || reinterpret_cast<uintptr_t>(p) % esz) return true;
  cudaPointerAttributes attr{};
  if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    cudaGetLastError();
    return true;
  }
  return (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) || attr.device != device;
}

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
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return report(ZERO_ECUDA, "no CUDA device");
  const int esz = c->dtype == ZERO_GRAD_FP32 ? 4 : 2, gsz = c->gain_dtype == ZERO_GRAD_FP32 ? 4 : 2;
  const zero_heads* in[2] = {q, k};
  const zero_heads* out[2] = {q_out, k_out};
  const void* gain[2] = {q_gain, k_gain};
  const int heads[2] = {c->q_heads, c->k_heads};
  for (int w = 0; w < 2; ++w) {
    if (heads[w] == 0) continue;
    if (!in[w] || bad(in[w]->data, esz, dev)) return report(ZERO_EINVAL, w ? "k must be aligned device memory" : "q must be aligned device memory");
    if (!out[w] || bad(out[w]->data, esz, dev))
      return report(ZERO_EINVAL, w ? "k's output must be aligned device memory" : "q's output must be aligned device memory");
    if (in[w]->token_stride < 0 || in[w]->head_stride < 0 || out[w]->token_stride < 0 || out[w]->head_stride < 0)
      return report(ZERO_EINVAL, "a stride is negative");
    if (gain[w] && bad(gain[w], gsz, dev)) return report(ZERO_EINVAL, "a gain must be aligned device memory");
    a->x[w] = {in[w]->data, in[w]->token_stride, in[w]->head_stride};
    a->out[w] = {out[w]->data, out[w]->token_stride, out[w]->head_stride};
    a->gain[w] = gain[w];
  }
  if (c->rotary_dim > 0 && c->n_positions > 0 && bad(table, 4, dev))
    return report(ZERO_EINVAL, "table must be aligned device memory");
  if (positions && bad(positions, 4, dev)) return report(ZERO_EINVAL, "positions must be aligned device memory");
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
  const int ctas = zfs::qk_ctas(tokens * (cfg->q_heads + cfg->k_heads));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->dtype == ZERO_GRAD_FP32) zfs::qk_kernel<true, false><<<ctas, zfs::kQkThreads, 0, s>>>(a);
  else zfs::qk_kernel<false, false><<<ctas, zfs::kQkThreads, 0, s>>>(a);
  return zfs::launched("norm and rotation launch");
}

zero_status zero_qk_backward_workspace_bytes(const zero_qk_config* cfg, int64_t tokens, int64_t* bytes) {
  if (!bytes) return zfs::report(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_config(cfg, tokens);
  if (st != ZERO_OK) return st;
  *bytes = static_cast<int64_t>(zfs::qk_ctas(tokens * (cfg->q_heads + cfg->k_heads))) * 2 * cfg->head_dim * 4;
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
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return zfs::report(ZERO_ECUDA, "no CUDA device");
  const int dsz = dgain_dtype == ZERO_GRAD_FP32 ? 4 : 2;
  if ((dq_gain && zfs::bad(dq_gain, dsz, dev)) || (dk_gain && zfs::bad(dk_gain, dsz, dev)))
    return zfs::report(ZERO_EINVAL, "a gain gradient must be aligned device memory");
  zfs::QkArgs a{};
  const long long rows = tokens * (cfg->q_heads + cfg->k_heads);
  const int ctas = zfs::qk_ctas(rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows > 0) {
    st = zfs::fill(cfg, tokens, q, k, q_gain, k_gain, table, positions, dq, dk, &a);
    if (st != ZERO_OK) return st;
    const zero_heads* dy[2] = {dq_out, dk_out};
    const int heads[2] = {cfg->q_heads, cfg->k_heads};
    for (int w = 0; w < 2; ++w) {
      if (heads[w] == 0) continue;
      if (!dy[w] || zfs::bad(dy[w]->data, cfg->dtype == ZERO_GRAD_FP32 ? 4 : 2, dev))
        return zfs::report(ZERO_EINVAL, "an output gradient must be aligned device memory");
      if (dy[w]->token_stride < 0 || dy[w]->head_stride < 0) return zfs::report(ZERO_EINVAL, "a stride is negative");
      a.dy[w] = {dy[w]->data, dy[w]->token_stride, dy[w]->head_stride};
    }
    int64_t need = 0;
    zero_qk_backward_workspace_bytes(cfg, tokens, &need);
    if (zfs::bad(workspace, 16, dev)) return zfs::report(ZERO_EINVAL, "workspace must be 16-byte aligned device memory");
    if (workspace_bytes < need) return zfs::report(ZERO_EINVAL, "workspace is too small");
    a.partials = static_cast<float*>(workspace);
    if (cfg->dtype == ZERO_GRAD_FP32) zfs::qk_kernel<true, true><<<ctas, zfs::kQkThreads, 0, s>>>(a);
    else zfs::qk_kernel<false, true><<<ctas, zfs::kQkThreads, 0, s>>>(a);
    st = zfs::launched("norm and rotation backward launch");
    if (st != ZERO_OK) return st;
  }
  if (!dq_gain && !dk_gain) return ZERO_OK;
  a.dim = cfg->head_dim;
  a.dgain[0] = dq_gain;
  a.dgain[1] = dk_gain;
  a.dgain_fp32 = dgain_dtype == ZERO_GRAD_FP32;
  zfs::qk_gain_kernel<<<(2 * a.dim + zfs::kQkThreads - 1) / zfs::kQkThreads, zfs::kQkThreads, 0, s>>>(a, ctas);
  return zfs::launched("gain gradient launch");
}

}  // extern "C"
