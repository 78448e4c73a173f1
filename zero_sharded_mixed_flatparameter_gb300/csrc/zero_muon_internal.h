// Internal interface of the Newton-Schulz orthogonalisation and of the Muon
// step (zero_orthogonalize.cpp, zero_muon_kernels.cu, zero_ns_gemm.cu).  Not
// part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "zero_internal.h"

struct zero_ns_config;

namespace zfs {

// Matrices of one launch (one shape); more of a shape go in several.
constexpr int kMaxMats = 64;
// Elements of one partial sum of a matrix's squared Frobenius norm.  The
// chunks are relative to the matrix and every thread takes the same elements
// whatever their alignment, so the norm does not depend on where a layout
// puts the matrix.
constexpr long long kNsChunk = 16384;

// ---- the orthogonalisation engine ------------------------------------------
// One stack of `mats` matrices of r x c.  m is the smaller side, n the larger.
// X is kept in the given orientation as fp16 with a power-of-two scale (see
// ns_gemm), pitch ldx; the Gram matrix A and the polynomial P are m x m,
// pitch ldm.
struct NsPlan {
  long long rows = 0, cols = 0;
  long long m = 0, n = 0;
  bool tall = false;       // rows > cols
  int mats = 0;            // matrices in flight (workspace)
  long long ldx = 0, ldm = 0;
  long long chunks = 0;    // norm partials per matrix
  // byte offsets in the workspace
  long long partials = 0, x_hi[2] = {0, 0}, x_lo[2] = {0, 0}, gram = 0, poly = 0, update = 0, bytes = 0;
};

// Where the finished stack goes.
struct NsOut {
  // Orthogonalised matrices as bf16 (out != nullptr), ...
  uint16_t* out = nullptr;
  long long row_stride = 0, mat_stride = 0;
  // ... or the Muon update of the flat buffer: w = w * decay - step * O.
  float* master = nullptr;
  uint16_t* p16 = nullptr;
  float decay = 1.0f, step = 0.0f;
  long long total_padded = 0;      // elements of master / p16 (debug bounds checks)
  const long long* dev_t = nullptr;  // capturable steps: nothing is written once *dev_t >= dev_steps
  long long dev_steps = 0;
  long long offset[kMaxMats] = {};
};

// The layout for `mats` matrices at once; `keep_update`: room for the fp32
// update (the Muon step's momentum pass writes it, the scale pass reads it).
NsPlan ns_plan(long long rows, long long cols, int mats, bool keep_update);
// How many of `batch` equal matrices one pass works on.
int ns_mats(long long rows, long long cols, long long batch);
// Checks steps, coefficients and eps; the reason in `why`.
bool ns_config_ok(const zero_ns_config& cfg, const char** why);
// Stacks that go through the steps together.
constexpr int kMaxProblems = 12;
// Elements of X that are worked on at once.
constexpr long long kNsBatch = 1LL << 27;
// A stack of as many is not put together with others: it fills the GPU (8 or
// more rounds of tiles), and a launch of several stacks looks up each tile's
// (the hidden-2048 model: 15.9 ms together, 15.5 apart; the hidden-1024 model,
// whose stacks are smaller: 1.94 and 2.29).
constexpr long long kNsAlone = 1LL << 26;
struct NsProblem;
// A problem's source, with its norm partials in the workspace, normalised.
cudaError_t ns_start(const NsProblem& q, const zero_ns_config& cfg, cudaStream_t stream, int* launches);
// The steps of all problems, from there to their `out`.
cudaError_t ns_run(const NsProblem* problems, int count, const zero_ns_config& cfg, cudaStream_t stream, int* launches);

// ---- elementwise passes (zero_muon_kernels.cu) -----------------------------
// A stack of strided matrices as the orthogonalisation's input.
struct MatSource {
  const void* data;
  int fp32;                 // else bf16
  long long row_stride, mat_stride;
  int vec_ok;               // 8-element vectors of a row are aligned
};
struct NsProblem {
  NsPlan plan;
  int mats;
  MatSource src;
  char* ws;
  NsOut out;
};
// Partial sums of squares, [mat][chunk].
cudaError_t launch_ns_norm(const MatSource& s, const NsPlan& p, int mats, double* partials, cudaStream_t stream);
// X0 = source / (norm + eps) as scaled fp16 pair (hi, lo).
struct ScaleArgs {
  MatSource src;
  long long rows, cols, ldx;
  int mats;
  int per_thread;           // vectors
  long long chunks;
  const double* partials;
  double eps;
  float scale;              // power of two of the stored values
  uint16_t* hi;             // fp16 bits, [mat][row][ldx]
  uint16_t* lo;             // or nullptr
};
cudaError_t launch_ns_scale(ScaleArgs a, cudaStream_t stream);

// The Muon step's momentum pass over up to kMaxMats equal matrices of the flat
// buffer: g = rank-order sum x 1/N x clip, mom = mu mom + g, update = nesterov
// ? g + mu mom : mom (fp32, [mat][numel]), and the norm partials of the update.
struct MomentumArgs {
  int n_ranks, grad_fp32, nesterov, mats;
  float inv_n, mu;
  const float* clip;
  unsigned long long* nonfinite;
  const long long* dev_t;
  long long dev_steps;
  long long numel, chunks;
  long long total_padded;
  float* mom;               // exp_avg of the flat buffer
  float* update;
  double* partials;
  long long offset[kMaxMats];
  const void* g[kMaxMats][kMaxRanks];  // the matrix's gradients, replica by replica
};
// `follows`: as with launch_ns_thin.
cudaError_t launch_momentum(const MomentumArgs& a, bool vec, bool follows, cudaStream_t stream);
unsigned int muon_debug_failures();

// ---- thin matrices (zero_ns_thin.cu) ---------------------------------------
// A smaller side of at most kThin: one launch for the whole orthogonalisation
// (and, in a Muon step, for its momentum pass and update), matrices of several
// shapes together.
constexpr int kThin = 128;
constexpr int kMaxSteps = 32;
// Bytes of the workspace that one launch may take (more only for a single
// matrix that needs more).
constexpr long long kThinWork = 1LL << 26;
// Factors of a step: the coefficients, and the powers of two between the
// stored (fp16) X, A and P.
struct ThinStep {
  float x;          // X as stored
  float gram;       // A from X X^T
  float square, gram_term, identity;  // P from A A, from A and on its diagonal
  float result;     // P X to the next X as stored (the last step: to its value)
};
struct ThinArgs {
  int steps;
  float eps;
  ThinStep step_factors[kMaxSteps];
  int rows[kMaxMats], cols[kMaxMats];  // a stack uses entry 0
  char* work;                          // thin_work() bytes per matrix
  long long work_mat_stride;           // of a stack
  // A stack: input and bf16 output.
  MatSource src;
  uint16_t* out;
  long long out_row_stride, out_mat_stride;
  int vec_out;
  // The Muon step: see MomentumArgs and NsOut.
  int n_ranks, grad_fp32, nesterov;
  float inv_n, mu, decay;
  const float* clip;
  unsigned long long* nonfinite;
  const long long* dev_t;
  long long dev_steps, total_padded;
  float *mom, *master;
  uint16_t* p16;
  uint32_t vec[(kMaxMats + 31) / 32];  // bit per matrix: 8-element vectors are aligned everywhere
  float step[kMaxMats];
  long long offset[kMaxMats], work_offset[kMaxMats];
  const void* g[kMaxMats][kMaxRanks];
};
// CTAs (a cluster) per matrix of this shape.
int thin_ctas(long long rows, long long cols);
// Bytes of workspace that a matrix of this shape needs (a multiple of 256).
long long thin_work(long long rows, long long cols, bool muon);
// Fills the scales and coefficients of `cfg`.
void thin_scales(const zero_ns_config& cfg, ThinArgs* a);
// `follows` (Muon): the launch before it belongs to the same step, and this one
// neither reads what that one writes nor writes what it uses; they may overlap.
cudaError_t launch_ns_thin(const ThinArgs& a, bool muon, bool follows, int ctas, long long mats, cudaStream_t stream,
                           int* launches);
unsigned int thin_debug_failures();
unsigned int thin_timeouts();

// ---- the products (zero_ns_gemm.cu) ----------------------------------------
enum NsEpilogue {
  kNsGram = 0,   // D = alpha acc, symmetric: only tiles on and below the diagonal are computed, both halves stored
  kNsPoly = 1,   // as kNsGram, D = alpha acc + cfactor C
  kNsApply = 2,  // D = alpha acc + cfactor (C + C_lo) as a pair (d_lo may be absent)
  kNsOut = 3,    // the finished matrices, likewise, as bf16
  kNsMuon = 4    // likewise, into the update of master and param16
};

struct GemmOperand {
  const uint16_t* data = nullptr;    // fp16 bits
  long long ld = 0, mat_stride = 0;  // elements
  bool k_major = true;  // element (i, k) at i * ld + k; else at k * ld + i
};

// C, C_lo, D and D_lo are fp16 with one layout (ldd, d_mat_stride); the powers
// of two of their scales are part of alpha and cfactor.
struct GemmArgs {
  long long M = 0, N = 0, K = 0;
  int mats = 0;
  GemmOperand a, b;
  int epilogue = kNsGram;
  float alpha = 1.0f, cfactor = 0.0f;
  const uint16_t* c = nullptr;
  const uint16_t* c_lo = nullptr;
  uint16_t* d = nullptr;
  uint16_t* d_lo = nullptr;
  long long ldd = 0, d_mat_stride = 0;
  NsOut out;
};
// One launch for `count` (up to kMaxProblems) stacks with one epilogue.
cudaError_t launch_ns_gemm(const GemmArgs* g, int count, cudaStream_t stream, int* launches);
unsigned int ns_gemm_debug_failures();
// Bounded waits of the products that gave up (0xFFFFFFFF if it cannot be read).
unsigned int ns_gemm_timeouts();

}  // namespace zfs
