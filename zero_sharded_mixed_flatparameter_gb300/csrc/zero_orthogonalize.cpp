// Newton-Schulz orthogonalisation of a stack of matrices: the host side.  It
// lays out the workspace, chooses the power-of-two scales of the fp16
// operands and enqueues the products; zero_orthogonalize is the public call,
// ns_run is shared with the Muon step (zero_runtime.cpp).
//
//   X0 = G / (|G|_F + eps)
//   A = X X^T,  P = a I + b A + c A A,  X <- P X      (steps times)
//
// with the products over the smaller side of G (X^T X and X P for a tall G):
// an odd polynomial of the singular values, whose vectors stay.  With the
// customary (3.4445, -4.7750, 2.0315) five steps bring every singular value
// that is not tiny to about 1.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

#include "zero_flatstep.h"
#include "zero_muon_internal.h"

namespace zfs {
namespace {

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

// Largest |p(s)| = |a s + b s^3 + c s^5| over 0 <= s <= top: at the end or
// where the derivative, a quadratic in s^2, vanishes.
double largest_value(double a, double b, double c, double top) {
  auto p = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
  double best = p(top);
  const double disc = 9.0 * b * b - 20.0 * a * c;
  double roots[2] = {-1.0, -1.0};
  if (c != 0.0) {
    if (disc >= 0.0) {
      roots[0] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
      roots[1] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
    }
  } else if (b != 0.0) {
    roots[0] = -a / (3.0 * b);
  }
  for (double t : roots)
    if (t > 0.0 && t < top * top) best = std::max(best, p(std::sqrt(t)));
  return best;
}

// Largest |b t + c t^2| over 0 <= t <= top: the spectral norm of P = b A + c A A.
double largest_factor(double b, double c, double top) {
  auto q = [&](double t) { return std::fabs(t * (b + t * c)); };
  double best = q(top);
  if (c != 0.0) {
    const double t = -b / (2.0 * c);
    if (t > 0.0 && t < top) best = std::max(best, q(t));
  }
  return best;
}

// The power of two that brings entries of a matrix of spectral norm `bound`
// (no entry is larger) to 2^14..2^15, half of what fp16 holds: 11 bits for
// every entry down to 2^-29 of the bound.
int scale_exponent(double bound) { return 15 - static_cast<int>(std::ceil(std::log2(std::max(bound, 1e-6) * 1.05))); }

constexpr double kLargestIterate = 1024.0;

// Steps whose X keeps its low half.  Noise that rounding puts into X at step k
// passes steps - k further polynomials, each of which multiplies the small
// singular values by up to a (3.4): with 11 bits alone a rank-1 matrix ends
// 1.5e-1 off after five steps (bf16: 1.2), with the low half kept until two
// polynomials are left 2.8e-3, and a Gaussian one 1.1e-3 either way.  (Larger a
// have few steps before the iterates outgrow their bound: 8.3 has two, and
// without a low half at all they end 1.7e-3 off, bf16's own rounding.)
int low_steps(int steps) { return std::max(steps - 2, 0); }

}  // namespace

bool ns_config_ok(const zero_ns_config& cfg, const char** why) {
  if (cfg.steps < 1 || cfg.steps > 32) {
    *why = "steps not in 1..32";
    return false;
  }
  if (!std::isfinite(cfg.a) || !std::isfinite(cfg.b) || !std::isfinite(cfg.c)) {
    *why = "coefficients must be finite";
    return false;
  }
  if (!std::isfinite(cfg.eps) || cfg.eps < 0.0f) {
    *why = "eps must be finite and >= 0";
    return false;
  }
  double top = 1.0;
  for (int k = 0; k < cfg.steps; ++k) {
    top = largest_value(cfg.a, cfg.b, cfg.c, top);
    if (!(top <= kLargestIterate)) {
      *why = "the coefficients let the iterates grow beyond 1024";
      return false;
    }
  }
  return true;
}

int ns_mats(long long rows, long long cols, long long batch) {
  const long long room = kNsBatch / std::max<long long>(rows * cols, 1);
  return static_cast<int>(std::max<long long>(1, std::min<long long>({batch, room, kMaxMats})));
}

NsPlan ns_plan(long long rows, long long cols, int mats, bool keep_update) {
  NsPlan p;
  p.rows = rows;
  p.cols = cols;
  p.tall = rows > cols;
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  p.mats = mats;
  p.ldx = round_up(cols, 16);  // rows of whole 32-byte sectors
  p.ldm = round_up(p.m, 16);
  p.chunks = (rows * cols + kNsChunk - 1) / kNsChunk;
  long long at = 0;
  auto take = [&](long long bytes) {
    const long long here = at;
    at = round_up(at + bytes, 256);
    return here;
  };
  p.partials = take(8 * p.chunks * mats);
  for (int k = 0; k < 2; ++k) {
    p.x_hi[k] = take(2 * p.ldx * rows * mats);
    p.x_lo[k] = take(2 * p.ldx * rows * mats);
  }
  p.gram = take(2 * p.ldm * p.m * mats);
  p.poly = take(2 * p.ldm * p.m * mats);
  if (keep_update) p.update = take(4 * rows * cols * mats);
  p.bytes = at;
  return p;
}

void thin_scales(const zero_ns_config& cfg, ThinArgs* a) {
  a->steps = cfg.steps;
  a->eps = cfg.eps;
  double top = 1.0;  // spectral norm of X
  for (int k = 0; k < cfg.steps; ++k) {
    ThinStep& f = a->step_factors[k];
    // P = a I + b A + c A A with its identity
    auto q = [&](double t) { return std::fabs(cfg.a + t * (cfg.b + t * cfg.c)); };
    double p = std::max(q(0.0), q(top * top));
    const double turn = cfg.c != 0.0f ? -cfg.b / (2.0 * cfg.c) : -1.0;
    if (turn > 0.0 && turn < top * top) p = std::max(p, q(turn));
    const double next = largest_value(cfg.a, cfg.b, cfg.c, top);
    const int ex = scale_exponent(top), ea = scale_exponent(top * top), ep = scale_exponent(p);
    f.x = std::ldexp(1.0f, ex);
    f.gram = std::ldexp(1.0f, ea - 2 * ex);
    f.square = cfg.c * std::ldexp(1.0f, ep - 2 * ea);
    f.gram_term = cfg.b * std::ldexp(1.0f, ep - ea);
    f.identity = cfg.a * std::ldexp(1.0f, ep);
    f.result = std::ldexp(1.0f, (k + 1 < cfg.steps ? scale_exponent(next) : 0) - ep - ex);
    top = next;
  }
}

// Matrices of a stack that one thin launch takes.
long long thin_mats(long long rows, long long cols, long long batch) {
  const long long each = thin_work(rows, cols, false);
  return std::max<long long>(1, std::min<long long>(batch, each > 0 ? kThinWork / each : 1 << 24));
}

cudaError_t ns_start(const NsProblem& q, const zero_ns_config& cfg, cudaStream_t stream, int* launches) {
  ScaleArgs s{};
  s.src = q.src;
  s.rows = q.plan.rows;
  s.cols = q.plan.cols;
  s.ldx = q.plan.ldx;
  s.mats = q.mats;
  s.chunks = q.plan.chunks;
  s.partials = reinterpret_cast<const double*>(q.ws + q.plan.partials);
  s.eps = cfg.eps;
  s.scale = std::ldexp(1.0f, scale_exponent(1.0));
  s.hi = reinterpret_cast<uint16_t*>(q.ws + q.plan.x_hi[0]);
  s.lo = low_steps(cfg.steps) > 0 ? reinterpret_cast<uint16_t*>(q.ws + q.plan.x_lo[0]) : nullptr;
  ++*launches;
  return launch_ns_scale(s, stream);
}

cudaError_t ns_run(const NsProblem* problems, int count, const zero_ns_config& cfg, cudaStream_t stream,
                   int* launches) {
  const int lows = low_steps(cfg.steps);
  double top = 1.0;  // bound of the spectral norm of X
  int ex = scale_exponent(top);
  for (int k = 0; k < cfg.steps; ++k) {
    const int from = k % 2, to = 1 - from;
    const bool low = k < lows, last = k + 1 == cfg.steps;
    const int ea = scale_exponent(top * top);
    const int ep = scale_exponent(largest_factor(cfg.b, cfg.c, top * top));
    const double next = largest_value(cfg.a, cfg.b, cfg.c, top);
    const int en = scale_exponent(next);
    GemmArgs gram[kMaxProblems], poly[kMaxProblems], apply[kMaxProblems];
    for (int i = 0; i < count; ++i) {
      const NsProblem& q = problems[i];
      const NsPlan& p = q.plan;
      auto half = [&](long long at) { return reinterpret_cast<uint16_t*>(q.ws + at); };
      GemmOperand x;
      x.data = half(p.x_hi[from]);
      x.ld = p.ldx;
      x.mat_stride = p.rows * p.ldx;
      GemmOperand square;
      square.ld = p.ldm;
      square.mat_stride = p.m * p.ldm;

      GemmArgs& g = gram[i];
      g.M = g.N = p.m;
      g.K = p.n;
      g.mats = q.mats;
      g.a = g.b = x;
      g.a.k_major = g.b.k_major = !p.tall;
      g.epilogue = kNsGram;
      g.alpha = std::ldexp(1.0f, ea - 2 * ex);
      g.d = half(p.gram);
      g.ldd = p.ldm;
      g.d_mat_stride = square.mat_stride;

      GemmArgs& s = poly[i];
      s.M = s.N = s.K = p.m;
      s.mats = q.mats;
      s.a = s.b = square;
      s.a.data = s.b.data = half(p.gram);
      s.epilogue = kNsPoly;
      s.alpha = cfg.c * std::ldexp(1.0f, ep - 2 * ea);
      s.cfactor = cfg.b * std::ldexp(1.0f, ep - ea);
      s.c = half(p.gram);
      s.d = half(p.poly);
      s.ldd = p.ldm;
      s.d_mat_stride = square.mat_stride;

      GemmArgs& u = apply[i];
      u.M = p.rows;
      u.N = p.cols;
      u.K = p.m;
      u.mats = q.mats;
      square.data = half(p.poly);
      if (p.tall) {  // X' = a X + X P, P symmetric
        u.a = x;
        u.b = square;
      } else {       // X' = a X + P X
        u.a = square;
        u.b = x;
        u.b.k_major = false;
      }
      const int eo = last ? 0 : en;
      u.alpha = std::ldexp(1.0f, eo - ex - ep);
      u.cfactor = cfg.a * std::ldexp(1.0f, eo - ex);
      u.c = x.data;
      u.c_lo = low ? half(p.x_lo[from]) : nullptr;
      u.ldd = p.ldx;
      u.d_mat_stride = x.mat_stride;
      if (last) {
        u.epilogue = q.out.out ? kNsOut : kNsMuon;
        u.out = q.out;
      } else {
        u.epilogue = kNsApply;
        u.d = half(p.x_hi[to]);
        u.d_lo = k + 1 < lows ? half(p.x_lo[to]) : nullptr;
      }
    }
    for (const GemmArgs* phase : {gram, poly, apply}) {
      const cudaError_t e = launch_ns_gemm(phase, count, stream, launches);
      if (e != cudaSuccess) return e;
    }
    top = next;
    ex = en;
  }
  return cudaSuccess;
}

namespace {

zero_status report(zero_status st, const char* fmt, long long x = 0, long long y = 0) {
  char buf[256];
  std::snprintf(buf, sizeof buf, fmt, x, y);
  zfs_report_error(nullptr, st, buf);
  return st;
}

zero_status check_shape(const zero_ns_config* cfg, int64_t rows, int64_t cols, int64_t batch) {
  if (!cfg) return report(ZERO_EINVAL, "config is NULL");
  const char* why = nullptr;
  if (!ns_config_ok(*cfg, &why)) return report(ZERO_EINVAL, why);
  if (rows < 0 || cols < 0 || batch < 0) return report(ZERO_EINVAL, "rows, cols and batch must not be negative");
  if (rows > (1LL << 30) || cols > (1LL << 30) || (cols > 0 && rows > (1LL << 40) / cols))
    return report(ZERO_EINVAL, "a matrix of %lld x %lld is too large", rows, cols);
  return ZERO_OK;
}

bool on_device(const void* p, int device) {
  cudaPointerAttributes attr{};
  if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) && attr.device == device;
}

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace zfs

extern "C" {

zero_status zero_orthogonalize_workspace_bytes(const zero_ns_config* cfg, int64_t rows, int64_t cols, int64_t batch,
                                               int64_t* bytes) {
  if (!bytes) return zfs::report(ZERO_EINVAL, "bytes is NULL");
  const zero_status st = zfs::check_shape(cfg, rows, cols, batch);
  if (st != ZERO_OK) return st;
  *bytes = rows == 0 || cols == 0 || batch == 0 ? 0
           : std::min(rows, cols) <= zfs::kThin
               ? zfs::thin_work(rows, cols, false) * zfs::thin_mats(rows, cols, batch)
               : zfs::ns_plan(rows, cols, zfs::ns_mats(rows, cols, batch), false).bytes;
  return ZERO_OK;
}

zero_status zero_orthogonalize(const zero_ns_config* cfg, int64_t rows, int64_t cols, int64_t batch, const void* in,
                               int32_t in_dtype, int64_t in_row_stride, int64_t in_batch_stride, void* out,
                               int64_t out_row_stride, int64_t out_batch_stride, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  zero_status st = zfs::check_shape(cfg, rows, cols, batch);
  if (st != ZERO_OK) return st;
  if (in_dtype != ZERO_GRAD_BF16 && in_dtype != ZERO_GRAD_FP32)
    return zfs::report(ZERO_EINVAL, "in_dtype %lld is neither bf16 (0) nor fp32 (1)", in_dtype);
  if (rows == 0 || cols == 0 || batch == 0) return ZERO_OK;
  if (in_row_stride < cols || out_row_stride < cols)
    return zfs::report(ZERO_EINVAL, "a row stride is below the %lld columns", cols);
  if (in_batch_stride < 0 || out_batch_stride < 0) return zfs::report(ZERO_EINVAL, "a batch stride is negative");
  if (batch > 1 && out_batch_stride < (rows - 1) * out_row_stride + cols)
    return zfs::report(ZERO_EINVAL, "out's batch stride makes its matrices overlap");
  const int esz = in_dtype == ZERO_GRAD_FP32 ? 4 : 2;
  int dev = -1;
  const cudaError_t got = cudaGetDevice(&dev);
  if (got != cudaSuccess) return zfs::report(ZERO_ECUDA, "no CUDA device");
  if (!in || zfs::misaligned(in, esz) || !zfs::on_device(in, dev))
    return zfs::report(ZERO_EINVAL, "in must be aligned memory of the current device");
  if (!out || zfs::misaligned(out, 2) || !zfs::on_device(out, dev))
    return zfs::report(ZERO_EINVAL, "out must be aligned memory of the current device");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto failed = [](cudaError_t e) {
    char buf[256];
    std::snprintf(buf, sizeof buf, "orthogonalize launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    zfs_report_error(nullptr, ZERO_ECUDA, buf);
    return ZERO_ECUDA;
  };
  auto source = [&](int64_t first) {
    zfs::MatSource src{};
    src.data = static_cast<const char*>(in) + first * in_batch_stride * esz;
    src.fp32 = in_dtype == ZERO_GRAD_FP32 ? 1 : 0;
    src.row_stride = in_row_stride;
    src.mat_stride = in_batch_stride;
    src.vec_ok = cols % zfs::kVec == 0 && in_row_stride % zfs::kVec == 0 && in_batch_stride % zfs::kVec == 0 &&
                 !zfs::misaligned(src.data, 16);
    return src;
  };
  int launches = 0;
  int64_t need = 0;
  zero_orthogonalize_workspace_bytes(cfg, rows, cols, batch, &need);
  if (need > 0 && (!workspace || zfs::misaligned(workspace, 256) || !zfs::on_device(workspace, dev)))
    return zfs::report(ZERO_EINVAL, "workspace must be 256-byte aligned memory of the current device");
  if (workspace_bytes < need)
    return zfs::report(ZERO_EINVAL, "workspace has %lld bytes, %lld needed", workspace_bytes, need);
  if (std::min(rows, cols) <= zfs::kThin) {
    zfs::ThinArgs a{};
    a.work = static_cast<char*>(workspace);
    a.work_mat_stride = zfs::thin_work(rows, cols, false);
    zfs::thin_scales(*cfg, &a);
    a.rows[0] = static_cast<int>(rows);
    a.cols[0] = static_cast<int>(cols);
    a.out_row_stride = out_row_stride;
    a.out_mat_stride = out_batch_stride;
    a.vec_out = out_row_stride % zfs::kVec == 0 && out_batch_stride % zfs::kVec == 0 && !zfs::misaligned(out, 16);
    const int64_t most = zfs::thin_mats(rows, cols, batch);
    for (int64_t first = 0; first < batch; first += most) {
      a.src = source(first);
      a.out = static_cast<uint16_t*>(out) + first * out_batch_stride;
      const cudaError_t e = zfs::launch_ns_thin(a, false, false, zfs::thin_ctas(rows, cols), std::min(most, batch - first), s,
                                                &launches);
      if (e != cudaSuccess) return failed(e);
    }
    return ZERO_OK;
  }
  const int mats = zfs::ns_mats(rows, cols, batch);
  const zfs::NsPlan p = zfs::ns_plan(rows, cols, mats, false);
  char* ws = static_cast<char*>(workspace);
  for (int64_t first = 0; first < batch; first += mats) {
    zfs::NsProblem q{};
    q.plan = p;
    q.mats = static_cast<int>(std::min<int64_t>(mats, batch - first));
    q.src = source(first);
    q.ws = ws;
    q.out.out = static_cast<uint16_t*>(out) + first * out_batch_stride;
    q.out.row_stride = out_row_stride;
    q.out.mat_stride = out_batch_stride;
    cudaError_t e = zfs::launch_ns_norm(q.src, p, q.mats, reinterpret_cast<double*>(ws + p.partials), s);
    if (e == cudaSuccess) e = zfs::ns_start(q, *cfg, s, &launches);
    if (e == cudaSuccess) e = zfs::ns_run(&q, 1, *cfg, s, &launches);
    if (e != cudaSuccess) return failed(e);
  }
  return ZERO_OK;
}

}  // extern "C"
