/*
 * zero_flatstep.h — C ABI of the GB300 (sm_103a) ZeRO-1/2/3 optimizer step
 * over a flattened, padded 1-D FlatParameter, with N data-parallel replicas
 * simulated on one GPU.
 *
 * The calls follow the ShardingStrategy protocol of Femtotron dev log #6
 * ("ZeRO-1 and ZeRO-2: abstraction design", section "ShardingStrategy as a
 * first-class abstraction"): make_master / reduce_grads / gather_weights /
 * post_step are the four points where ZeRO enters a training step, with the
 * optimizer step between reduce_grads and gather_weights.  Plain data
 * parallelism (stage 0, "NoShard") runs through the same calls.
 *
 * Conventions for every call:
 *  - Plain pointers and sizes only.  "dev" pointers are CUDA device memory
 *    owned by the caller; the library never allocates, frees or retains
 *    device memory, and holds only host-side metadata in a zero_ctx.  Two
 *    stated exceptions: zero_clip_grad_norm_static's fixed scratch array in
 *    the library's own device memory, and an offload context's host worker
 *    threads (see the ZeRO-Offload calls).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Device work is enqueued on it asynchronously; the caller keeps
 *    every buffer alive until that work has completed on the stream.  The
 *    ZeRO-3 gathers and the clip norm pass are launched with programmatic
 *    stream serialization: their thread blocks may become resident while the
 *    kernel before them on the stream finishes, but each waits for that
 *    kernel to complete (and its writes to be visible) before it reads
 *    anything, so the stream's ordering is the usual one.
 *  - Every call returns a zero_status; nothing crosses the ABI as an
 *    exception.  A call that fails leaves the context unchanged.  The text of
 *    the last error is available from zero_last_error().
 *  - A context is not thread-safe: calls on one context must not overlap.
 */
#ifndef ZERO_FLATSTEP_H
#define ZERO_FLATSTEP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zero_status {
  ZERO_OK = 0,
  ZERO_EINVAL = 1,   /* invalid argument (null/misaligned pointer, bad size, bad config) */
  ZERO_ENOMEM = 2,   /* host allocation of metadata failed */
  ZERO_ECUDA = 3,    /* a CUDA runtime call or kernel launch failed */
  ZERO_ESTATE = 4,   /* call not allowed in the context's current state */
  ZERO_ENOTSUP = 5   /* valid request this build does not support */
} zero_status;

typedef enum zero_grad_dtype {
  ZERO_GRAD_BF16 = 0,  /* replica gradients are bf16 (2 bytes/element) */
  ZERO_GRAD_FP32 = 1   /* replica gradients are fp32 (fp32 gradient accumulation) */
} zero_grad_dtype;

/*
 * Optimizer and sharding configuration.
 *  stage       0 = plain data parallelism (no sharding, no padding), 1 = ZeRO-1
 *              (optimizer state sharded), 2 = ZeRO-2 (+ gradients), 3 = ZeRO-3
 *              (+ parameters) — CMU 15-779 Lecture 13 notes §3.1-3.3.
 *  n_ranks     N simulated data-parallel replicas, 1..16.
 *  grad_dtype  zero_grad_dtype of the replica gradient buffers.
 *  adamw       1 = decoupled weight decay (AdamW), 0 = Adam (weight_decay must be 0).
 *  lr, beta1, beta2, eps, weight_decay: fp32 Adam hyper-parameters
 *              (notes §2.1); beta1, beta2 in [0, 1), eps >= 0, lr finite.
 */
typedef struct zero_config {
  int32_t stage;
  int32_t n_ranks;
  int32_t grad_dtype;
  int32_t adamw;
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
} zero_config;

/*
 * Caller-allocated device buffers, each of `padded_numel` elements (see
 * zero_plan / zero_padded_numel) and 16-byte aligned:
 *  master      fp32 master weights (the optimizer's copy, notes §2.2)
 *  exp_avg     fp32 Adam first moment m
 *  exp_avg_sq  fp32 Adam second moment v
 *  param16     bf16 parameters.  Stages 0-2: the full compute copy every
 *              replica holds after the all-gather.  Stage 3: the rank-major
 *              shard storage (rank d's shard of unit i at base_i + d*shard_i),
 *              which has the same byte layout.
 */
typedef struct zero_buffers {
  float* master;
  float* exp_avg;
  float* exp_avg_sq;
  void* param16;
} zero_buffers;

typedef struct zero_ctx zero_ctx;

/*
 * zero_plan — FlatParameter layout only (host, no device work).
 * Lecture notes §0.4 and §5.2: each unit's parameters are flattened and
 * concatenated in caller order, right-padded with zeros to a multiple of the
 * shard count F (N for stages 1-3, 1 for stage 0) and split into F equal
 * shards; rank d owns shard d.  Femtotron dev log #6 ("master is sharded 1-D,
 * not by shape").
 *  param_numel[n_params]  element count of each parameter (>= 0)
 *  param_unit[n_params]   unit (FlatParameter) id of each parameter; ids are
 *                         nondecreasing and start at 0 (n_units = last id + 1;
 *                         a skipped id is an empty unit)
 *  out                    receives a context usable for layout / ledger queries;
 *                         step calls on it return ZERO_ESTATE.
 * Errors: ZERO_EINVAL for a bad config, negative sizes, decreasing unit ids or
 * null pointers with n_params > 0; ZERO_ENOMEM.
 */
zero_status zero_plan(const zero_config* cfg, const int64_t* param_numel, const int32_t* param_unit,
                      int32_t n_params, zero_ctx** out);

/*
 * zero_make_master — the protocol's make_master: plan the layout (as
 * zero_plan), then build the fp32 master from the caller's fp32 parameters:
 * copy parameter p (init_params[p], param_numel[p] fp32 device elements,
 * 4-byte aligned) to its flat offset, zero every pad, zero m and v, write
 * param16 = bf16(master) (round to nearest even) and set the step count t = 0.
 * Enqueued on `stream`; init_params may be released once it completes.
 * Errors: as zero_plan, plus ZERO_EINVAL for a null `bufs`, a null or
 * non-16-byte-aligned buffer, a null init pointer for a non-empty parameter,
 * or a pointer that is not device memory; ZERO_ECUDA on launch failure.
 */
zero_status zero_make_master(const zero_config* cfg, const int64_t* param_numel,
                             const int32_t* param_unit, int32_t n_params,
                             const float* const* init_params, const zero_buffers* bufs,
                             void* stream, zero_ctx** out);

/* Number of units; total padded and unpadded element counts. */
zero_status zero_num_units(const zero_ctx* ctx, int32_t* n_units);
zero_status zero_padded_numel(const zero_ctx* ctx, int64_t* padded, int64_t* numel);

/*
 * zero_layout — unit i's element count, padded count (multiple of F), shard
 * length (padded / F) and flat base offset (sum of earlier padded counts).
 * ZERO_EINVAL if unit is out of range.
 */
zero_status zero_layout(const zero_ctx* ctx, int32_t unit, int64_t* numel, int64_t* padded,
                        int64_t* shard, int64_t* base);

/* Flat offset of parameter p inside the padded buffer. */
zero_status zero_param_offset(const zero_ctx* ctx, int32_t param, int64_t* offset);

/*
 * zero_state_bytes — per-rank model-state bytes of this layout under `stage`
 * (lecture notes §2.3 and §9 item 2: bf16 params 2, bf16 grads 2, optimizer
 * state K = 12 bytes per element; stage 1 shards K, stage 2 also the grads,
 * stage 3 also the params): 16P, 4P + 12S, 2P + 14S, 16S with P the total
 * and S the per-rank shard total of the layout as `stage` pads it with the
 * context's N — no padding for stage 0, each unit padded to a multiple of N
 * for stages 1-3 (notes §3.6) — whatever stage the context itself runs (a
 * stage-0 context, which does not pad, still reports the shards a sharded
 * stage would hold).  per_rank_bytes has n_ranks entries.
 */
zero_status zero_state_bytes(const zero_ctx* ctx, int32_t stage, int64_t* per_rank_bytes);

/*
 * zero_stage3_peak_bytes — ZeRO-3 model-state peak of one rank during
 * backward (lecture notes §3.5 and §11 Exercise 5): resident shards, plus the
 * grad shards of units already reduce-scattered, plus the full bf16 params and
 * grads of the unit being processed (units processed last to first), each
 * unit padded to a multiple of N as stage 3 pads it.
 * peak_unit receives the unit where the peak occurs (-1 if none).
 */
zero_status zero_stage3_peak_bytes(const zero_ctx* ctx, int64_t* peak_bytes, int32_t* peak_unit);

/*
 * zero_reduce_grads — the protocol's reduce_grads (Femtotron dev log #7, the
 * ZeRO-2 post-accumulate-grad hook: flatten, zero-pad, reduce-scatter AVG).
 * Registers the N replicas' gradients of one unit (unit >= 0: N pointers to
 * padded_i elements each) or of the whole buffer (unit == -1: N pointers to
 * padded_numel elements each).  Pad entries must be zero, as the hook's zero
 * padding makes them.  The reduction itself — the rank-order fp32 sum scaled
 * by 1/N, the local stand-in for reduce-scatter — is fused into zero_step, so
 * this call does no device work; the buffers must stay valid and unchanged
 * until the zero_step that consumes them has completed on its stream.
 * Registering a unit again replaces its pointers.
 * Errors: ZERO_EINVAL (unit out of range, null pointer, pointer not aligned to
 * the element size); ZERO_ESTATE if no buffers are bound, a step is pending
 * its post_step, or a clip is pending (zero_clip_grad_norm ran on the
 * gradients registered before it: register every unit first, then clip).
 */
zero_status zero_reduce_grads(zero_ctx* ctx, int32_t unit, const void* const* replica_grads,
                              void* stream);

/*
 * zero_accumulate_grads — fp32 gradient accumulation of one micro-step
 * (Femtotron dev log #5: no_sync micro-steps accumulate before the single
 * reduce; the source guide's Megatron main_grad: fp32 accumulation, the
 * 18 B/param case).  For each replica r and element j of the unit (unit >= 0:
 * padded_i elements) or of the whole buffer (unit == -1: padded_numel):
 *   acc[r][j] = (first ? 0 : acc[r][j]) + float(micro[r][j])
 * one fp32 addition per micro-step, no scaling (scale the loss by
 * 1/accum_steps, as the pages do).  micro: N bf16 device buffers (2-byte
 * aligned); acc: N fp32 device buffers (4-byte aligned), caller-owned; both
 * 16-byte aligned for the vector kernel.  The accumulators are then
 * registered with zero_reduce_grads on a context whose grad_dtype is fp32.
 * Enqueued on `stream`; no context state changes.
 * Errors: ZERO_EINVAL (grad_dtype is not fp32, unit out of range, null or
 * misaligned pointer); ZERO_ESTATE (no buffers bound); ZERO_ECUDA.
 */
zero_status zero_accumulate_grads(zero_ctx* ctx, int32_t unit, const void* const* micro_grads_bf16,
                                  float* const* accumulators, int32_t first, void* stream);

/*
 * zero_step — one optimizer step, t <- t + 1, in one fused pass over the
 * padded flat buffer (lecture notes §2.1-§3.3; Femtotron dev logs #4/#5 step
 * order).  For every element j of every rank's shard:
 *   g  = ((G_0[j] + G_1[j]) + ... + G_{N-1}[j]) * (1/N)      fp32, rank order
 *   w  = w * (1 - lr*wd)                                      AdamW only
 *   m  = beta1*m + (1-beta1)*g;  v = beta2*v + (1-beta2)*g*g
 *   w  = w - lr * ((m / (1-beta1^t)) / (sqrt(v / (1-beta2^t)) + eps))
 *   param16[j] = bf16_rne(w)     (the all-gather's stand-in for stages 0-2)
 * Every operation is a separately rounded IEEE fp32 operation (no FMA
 * contraction, IEEE division and square root).  After zero_clip_grad_norm,
 * g is multiplied by the clip coefficient before Adam.  Requires every unit's
 * gradients registered since the last post_step.
 * In capturable mode (zero_enable_capturable) the bias corrections come
 * from the device table and one more one-thread launch advances the device
 * step count.
 * Errors: ZERO_ESTATE (no buffers, missing gradients, step already taken
 * without post_step, an offload context — its step is zero_offload_step);
 * ZERO_ECUDA (a launch failed; t is left unchanged, but
 * when a step needs more than one launch — more than 48 gradient segments, or
 * both aligned and unaligned ones — launches enqueued before the failing one
 * have updated their elements).
 */
zero_status zero_step(zero_ctx* ctx, void* stream);

/*
 * zero_clip_workspace_bytes — size of the device workspace zero_clip_grad_norm
 * needs for this layout: 32 bytes of header plus 8 bytes per norm chunk
 * (every unit is cut into chunks of 16,384 elements).
 */
zero_status zero_clip_workspace_bytes(const zero_ctx* ctx, int64_t* bytes);

/*
 * zero_count_nonfinite — overflow count of the step.  DeepSpeed's ZeRO step
 * checks the gradients for overflow before it clips and updates (source guide
 * §4.3); here the fused step counts, at no extra memory traffic, the elements
 * whose reduced gradient g = (sum of the N replicas, rank order, fp32) / N is
 * inf or NaN — a non-finite replica gradient or an fp32 overflow of the sum —
 * and adds that number to *counter.  Every later zero_step (and
 * zero_offload_step) of this context counts, clipped or not; the step is
 * taken all the same (the non-finite values propagate as IEEE arithmetic
 * makes them), so a caller that wants to skip such steps clips first and
 * reads zero_grad_norm, or restores a checkpoint when the count moves.
 *  counter  caller-owned device uint64_t, 8-byte aligned, on the context's
 *           device; the library adds to it and never clears it (the caller
 *           zeroes it, e.g. with cudaMemsetAsync, for a fresh count) and it
 *           must stay allocated while counting is on.  NULL stops counting.
 * Errors: ZERO_EINVAL (misaligned, host or other-device counter).
 */
zero_status zero_count_nonfinite(zero_ctx* ctx, uint64_t* counter);

/*
 * zero_read_nonfinite — waits for `stream` and copies the counter given to
 * zero_count_nonfinite into *count.  ZERO_ESTATE when no counter is set;
 * ZERO_ECUDA if the copy fails.
 */
zero_status zero_read_nonfinite(zero_ctx* ctx, uint64_t* count, void* stream);

/*
 * zero_clip_grad_norm — global-norm gradient clipping, the ClipGradNorm
 * transform Femtotron dev logs #4/#5 apply to the fp32 gradient before AdamW
 * (the source guide's --clip-grad 1.0 / gradient_clipping 1.0).  On `stream`
 * it computes the L2 norm of the reduced gradient g = (sum of the N
 * registered replicas) / N over every element of every unit, and the
 * coefficient c = min(1, max_norm / (norm + 1e-6)) rounded to fp32; the next
 * zero_step multiplies every reduced gradient by c before Adam.  Non-finite
 * gradients follow IEEE arithmetic and torch's clip_grad_norm_: an inf makes
 * the norm inf and c = 0 (the inf element becomes inf * 0 = NaN, every other
 * gradient 0); a NaN makes the norm NaN and c = NaN (every gradient NaN).  A
 * caller that skips such steps reads zero_grad_norm before zero_step.  The squared
 * norm is summed over fixed chunks of 16,384 elements of each unit (pads
 * included, they add zero) in a fixed order, so the result is reproducible
 * and identical for every stage and for padded or unpadded layouts.
 *  max_norm    > 0 and finite
 *  workspace   caller-allocated device scratch of at least
 *              zero_clip_workspace_bytes() bytes, 16-byte aligned, owned by the
 *              caller; it holds the norm and coefficient until the next clip
 *              and must stay allocated until that zero_step has completed.
 * Call after every unit's gradients are registered and before zero_step.
 * Errors: ZERO_EINVAL (bad max_norm, null/misaligned/small/host workspace);
 * ZERO_ESTATE (no buffers, gradients missing, step pending post_step);
 * ZERO_ECUDA.
 */
zero_status zero_clip_grad_norm(zero_ctx* ctx, float max_norm, void* workspace, int64_t workspace_bytes,
                                void* stream);

/*
 * Flag of zero_clip_grad_norm_ex / zero_clip_workspace_bytes_ex: keep the
 * reduced fp32 gradient in the workspace so that the next zero_step reads it
 * (4 bytes per element) instead of the N replicas (2N or 4N bytes): the
 * clipped step then moves 2N + 34 instead of 4N + 26 bytes per element (bf16
 * replicas), fewer for N > 4.  Results are bit-identical either way.
 */
#define ZERO_CLIP_KEEP_REDUCED 1

/* Workspace size of zero_clip_grad_norm_ex for `flags`: with
 * ZERO_CLIP_KEEP_REDUCED, plus 4 bytes per padded element (256-byte aligned). */
zero_status zero_clip_workspace_bytes_ex(const zero_ctx* ctx, int32_t flags, int64_t* bytes);

/*
 * zero_clip_grad_norm_ex — zero_clip_grad_norm with flags (0 or
 * ZERO_CLIP_KEEP_REDUCED).  With ZERO_CLIP_KEEP_REDUCED the workspace must
 * hold zero_clip_workspace_bytes_ex(ctx, ZERO_CLIP_KEEP_REDUCED) bytes and
 * stay allocated and unchanged until the next zero_step has completed; the
 * registered replica buffers are not read again by that step.
 * Errors: as zero_clip_grad_norm; ZERO_EINVAL for unknown flags.
 */
zero_status zero_clip_grad_norm_ex(zero_ctx* ctx, float max_norm, int32_t flags, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/*
 * zero_clip_grad_norm_static — zero_clip_grad_norm for callers that cannot
 * allocate device memory (for example code running inside an allocator or
 * an out-of-memory handler, or in a loop where allocation is forbidden), so
 * cannot hand in a workspace.  The pages have no counterpart: this is a
 * property of this library's interface, not of the method.
 * Same computation and result as zero_clip_grad_norm; the scratch is a fixed
 * 1 MiB array in the library's own device memory (one per CUDA context that
 * loads the library's device code — normally one per GPU — held until that
 * context ends), so layouts needing more than that — about 2.1e9 padded
 * elements — are rejected with ZERO_EINVAL.  The call allocates nothing.
 * Its first call in a CUDA context looks up the array's device address in
 * that context (set-up, once per context, keyed on the context's unique id,
 * so a second context on the same GPU or the primary context re-created
 * after cudaDeviceReset gets its own lookup); that first lookup may load the
 * library's device code into the context, which creates the array.  So make
 * the first call in each context before any stream capture and before any
 * region that must not allocate.  All calls in a context share the array
 * and it keeps the last call's contents: calls whose device work can overlap
 * race on it, and between a call and the same zero_ctx's zero_step no other
 * static-scratch clip may run unless all are ordered on one stream.
 * Errors: as zero_clip_grad_norm; ZERO_EINVAL when the layout is too large.
 */
zero_status zero_clip_grad_norm_static(zero_ctx* ctx, float max_norm, void* stream);

/*
 * zero_grad_norm — the norm computed by the last zero_clip_grad_norm on this
 * context, copied to the host.  Synchronizes `stream` (the stream the clip
 * ran on).  ZERO_ESTATE if no clip has run.
 */
zero_status zero_grad_norm(zero_ctx* ctx, double* norm, void* stream);

/*
 * zero_gather_weights — the protocol's gather_weights.  Stage 3 (ZeRO-3
 * unshard, lecture notes §3.3 and §5.1): copy unit `unit`'s N bf16 shards, in
 * rank order, into `unit_buf` (padded_i bf16 elements, device, 2-byte
 * aligned); unit == -1 copies the whole padded buffer.  Stages 0-2: the fused
 * step has already written every replica's full bf16 copy, so this returns
 * ZERO_OK without device work (unit_buf may be NULL).
 * Errors: ZERO_EINVAL (unit out of range, null/misaligned unit_buf at stage 3);
 * ZERO_ESTATE (no buffers bound); ZERO_ECUDA.
 */
zero_status zero_gather_weights(zero_ctx* ctx, int32_t unit, void* unit_buf, void* stream);

/*
 * zero_gather_units — zero_gather_weights for `count` consecutive units
 * first_unit .. first_unit + count - 1 at once: unit first_unit + k into
 * unit_bufs[k] (a host array of `count` device pointers, each padded_i bf16
 * elements, 2-byte aligned; NULL allowed only for empty units).  The
 * ZeRO-3 prefetch of the source guide's DeepSpeed section (the parameter
 * coordinator gathers the next modules' parameters ahead of use, several
 * parameters coalesced into one collective) and Megatron's bucket-by-bucket
 * parameter all-gather: the copies are those of zero_gather_weights, issued
 * as one kernel per 32 units instead of one per unit.  The buffers must not
 * overlap one another or the parameter storage.  count == 0 and stages 0-2:
 * ZERO_OK without device work (unit_bufs may be NULL).
 * Errors: ZERO_EINVAL (count < 0, units out of range, null unit_bufs, null
 * or misaligned buffer of a non-empty unit at stage 3); ZERO_ESTATE (no
 * buffers bound); ZERO_ECUDA.
 */
zero_status zero_gather_units(zero_ctx* ctx, int32_t first_unit, int32_t count, void* const* unit_bufs,
                              void* stream);

/*
 * zero_post_step — the protocol's post_step: forget the registered gradients
 * (and the pending clip coefficient) so the next step needs fresh ones.
 * ZERO_ESTATE unless a step was taken since the last post_step.  No device
 * work.
 */
zero_status zero_post_step(zero_ctx* ctx, void* stream);

/*
 * zero_export_state — checkpoint the optimizer state in a layout-free form
 * (lecture notes §5.2: the pads are not parameters): the real elements of
 * master, m and v, unit by unit with the pads dropped — i.e. the parameters
 * back to back in caller order, numel_total elements per array — into
 * caller-allocated device fp32 buffers (4-byte aligned), and the step count
 * into *t.  Any context planned over the same parameter list, with any N,
 * stage or unit grouping of the same order, can import it (resharding; the
 * source guide's resharding checkpoints, Femtotron #5's dp_size change).
 * Enqueued on `stream` (in an offload context: copies up from the host state,
 * which must not change until they complete).  Errors: ZERO_EINVAL
 * (null/misaligned/host pointer); ZERO_ESTATE (no buffers); ZERO_ECUDA.
 */
zero_status zero_export_state(zero_ctx* ctx, float* master_out, float* exp_avg_out, float* exp_avg_sq_out,
                              int64_t* t, void* stream);

/*
 * zero_import_state — restore state exported by zero_export_state (from this
 * or any other layout of the same parameters): master, m and v are written
 * into this context's padded layout with zero pads, param16 = bf16(master)
 * (round to nearest even), and the step count set to t.  Not allowed while
 * a step awaits its post_step.  Enqueued on `stream`; the inputs may be
 * released once it completes (in an offload context the host state is
 * written and the call synchronizes `stream`).  Errors: ZERO_EINVAL
 * (null/misaligned/host pointer, t < 0); ZERO_ESTATE; ZERO_ECUDA.
 */
zero_status zero_import_state(zero_ctx* ctx, const float* master_in, const float* exp_avg_in,
                              const float* exp_avg_sq_in, int64_t t, void* stream);

/* ---- Capturable steps (CUDA graphs) --------------------------------------
 * The pages have no counterpart: this is the library's way of letting a
 * whole step (registration, clip, step, post_step, gathers) be captured once
 * into a CUDA graph and replayed every iteration without host work.  A
 * replayed launch repeats its arguments, so what changes from step to step
 * (the bias corrections 1 - beta^t) must come from device memory: in
 * capturable mode the step count lives on the device and the kernels look up
 * bc1, bc2 of step t in a table the host computed once (the same fp32 values
 * zero_step would pass, so results are bit-identical).  Each zero_step (and
 * each replay of a captured one) reads the count, updates, and then advances
 * the count with one extra one-thread launch.  Replays also repeat the
 * gradient pointers, the clip workspace and the learning rate captured.
 */

/* Bytes of the capturable workspace for up to max_steps steps in total
 * (16 + 8 * max_steps).  Errors: ZERO_EINVAL. */
zero_status zero_capturable_workspace_bytes(const zero_ctx* ctx, int64_t max_steps, int64_t* bytes);

/*
 * zero_enable_capturable — turn the mode on: workspace = device memory of the
 * context's device (16-byte aligned, caller-owned, kept until
 * zero_disable_capturable), holding the step count (set to the steps taken
 * so far) and the bias corrections of steps 1..max_steps.  Synchronizes
 * `stream`.  A step whose count would pass max_steps is skipped by the
 * kernels (nothing changes; zero_step_count then reports ZERO_ESTATE).
 * Errors: ZERO_EINVAL (workspace, max_steps <= steps taken); ZERO_ESTATE (a
 * step awaits post_step); ZERO_ENOTSUP (offload context); ZERO_ENOMEM;
 * ZERO_ECUDA.  Export and import are refused while the mode is on.
 */
zero_status zero_enable_capturable(zero_ctx* ctx, void* workspace, int64_t workspace_bytes, int64_t max_steps,
                                   void* stream);

/*
 * zero_disable_capturable — turn the mode off: the context's step count
 * becomes the device count (capped at max_steps: later steps were skipped).
 * Synchronizes `stream`.  Errors: ZERO_ESTATE (mode not on); ZERO_ECUDA.
 */
zero_status zero_disable_capturable(zero_ctx* ctx, void* stream);

/* ---- ZeRO-Offload -------------------------------------------------------
 * CMU 15-779 Lecture 13 notes §7.1-7.2 (ZeRO-Offload's partition and its
 * timeline): only the 16-bit parameters stay on the GPU; the fp32 master,
 * m and v live in host memory and a multi-threaded CPU Adam updates them
 * chunk by chunk while the GPU produces the next chunk's gradient, the new
 * bf16 parameters going back up chunk by chunk.  Here the gradient that goes
 * down is the reduced fp32 one (sum of the N replicas in rank order x 1/N,
 * times a pending clip coefficient): the host update is the device step's
 * arithmetic, bit for bit, so an offloaded run equals a GPU-resident one.
 */

/*
 * zero_make_master_offload — zero_make_master for an offload context:
 * bufs->master, exp_avg, exp_avg_sq are HOST memory (pageable or pinned,
 * padded_numel floats each, 16-byte aligned, caller-owned), bufs->param16 is
 * device memory as before; init_params are device fp32 buffers.  The host
 * master gets the init params at their offsets (pads, m, v zero), param16 =
 * bf16(init) on the device.  Synchronizes `stream`.  The context then steps
 * with zero_offload_step only (zero_step returns ZERO_ESTATE); registration,
 * clipping (without ZERO_CLIP_KEEP_REDUCED: ZERO_ENOTSUP), accumulation,
 * gather, export/import and post_step work as for any context.
 * Errors: as zero_make_master, plus ZERO_EINVAL for a device state buffer.
 */
zero_status zero_make_master_offload(const zero_config* cfg, const int64_t* param_numel,
                                     const int32_t* param_unit, int32_t n_params,
                                     const float* const* init_params, const zero_buffers* bufs,
                                     void* stream, zero_ctx** out);

/*
 * zero_offload_workspace_bytes — sizes of the two workspaces of
 * zero_offload_step for chunks of `chunk` elements: *host_bytes of pinned
 * host memory (3 chunk slots of fp32 gradient + bf16 parameters) and
 * *device_bytes of device memory (3 slots of fp32 gradient).
 * Errors: ZERO_EINVAL (NULL, chunk < 1).
 */
zero_status zero_offload_workspace_bytes(const zero_ctx* ctx, int64_t chunk, int64_t* host_bytes,
                                         int64_t* device_bytes);

/*
 * zero_offload_step — one optimizer step of an offload context, t += 1.  The
 * padded buffer is processed in chunks of `chunk` elements through a ring of
 * 3 workspace slots: on `stream` a kernel writes chunk c's reduced (clipped)
 * fp32 gradient into a device slot and it is copied to a pinned host slot;
 * the host waits for it, runs Adam / AdamW over the chunk's host master, m, v
 * on n_threads threads (0: one per hardware thread; the calling thread is one
 * of them), writing bf16 parameters into a host slot that is copied into
 * param16 on `copy_stream` (NULL: `stream`) — so the GPU reduction and the
 * copies of other chunks overlap each chunk's host update.  param16 is
 * rewritten only after the work enqueued on `stream` before the call, and
 * work enqueued on `stream` after it sees the new param16.  Blocks the
 * calling thread until every chunk's host update is done.  Workspaces: see
 * zero_offload_workspace_bytes; host_workspace must be page-locked,
 * device_workspace memory of the context's device, both 16-byte aligned.
 * Not thread-safe on one context.  Errors: ZERO_EINVAL (chunk, threads,
 * workspaces); ZERO_ESTATE (not an offload context, unregistered unit,
 * step pending post_step); ZERO_ENOMEM (threads cannot start); ZERO_ECUDA
 * (the chunks done before the failure stay updated on the host).
 */
zero_status zero_offload_step(zero_ctx* ctx, int64_t chunk, void* host_workspace, int64_t host_bytes,
                              void* device_workspace, int64_t device_bytes, int32_t n_threads,
                              void* stream, void* copy_stream);

/*
 * zero_cpu_adam — the CPU Adam of the offload step on its own, over host
 * arrays of n elements: given the reduced fp32 gradient `grad`, updates
 * master, exp_avg, exp_avg_sq in place with step t (>= 1) of cfg's
 * optimizer and writes param16 = bf16(master) (bit patterns, round to
 * nearest even).  Same arithmetic as the device step.  n_threads as above;
 * the threads belong to one process-wide pool kept between calls (calls from
 * several threads take turns).  No CUDA call is made.
 * Errors: ZERO_EINVAL (config, t < 1, n < 0, NULL or misaligned pointer);
 * ZERO_ENOMEM.
 */
zero_status zero_cpu_adam(const zero_config* cfg, int64_t t, const float* grad, float* master,
                          float* exp_avg, float* exp_avg_sq, uint16_t* param16, int64_t n,
                          int32_t n_threads);

/* ---- Muon: orthogonalised updates of the matrices -------------------------
 * The pages stop at Adam; this is the optimizer step for a model whose
 * matrices take an orthogonalised momentum update while everything else
 * (embeddings, norms, biases, heads) stays with Adam / AdamW in the same
 * zero_step.  A shard boundary may cut a matrix anywhere, so the update needs
 * the whole matrix; all shards of the simulated ranks live in one buffer, and
 * the result does not depend on the stage (bit for bit: the matrices of a
 * context, which do count, are the same; see zero_orthogonalize).
 */

/*
 * Newton-Schulz orthogonalisation of a matrix G:
 *   X = G / (|G|_F + eps), then `steps` times
 *   X <- a X + b (X X^T) X + c (X X^T)^2 X
 * an odd polynomial of the singular values that leaves the singular vectors.
 * Precision: fp32 sums of products of fp16 operands with power-of-two scales,
 * 11 bits (22 for X while later steps still amplify its rounding); 22 bits
 * throughout where the smaller side is at most 128.  Error of the bf16 result
 * against exact arithmetic, relative to its norm and bf16's own 1.7e-3 included,
 * for the customary (3.4445, -4.7750, 2.0315): 2.3e-3 after 5 steps on matrices
 * of full rank and 3.3e-3 on low ranks, 3.7e-3 after 8 steps (smaller sides up to
 * 128: 1.7e-3, and 2.2e-3 on low ranks after 8 steps).  Beyond, or
 * with a larger a, rounding noise outside a low rank grows by up to |a| a step, as
 * it does in fp32 (10 steps: 2.4e-2, fp32 4.3e-2); and coefficients whose terms
 * nearly cancel magnify what was rounded (4.0848, -6.8946, 2.9270 at a singular
 * value of 1: 7.5e-3 after one step).
 *  steps    1..32;  a, b, c, eps: finite, eps >= 0; coefficients under which
 *           a singular value in [0, 1] grows beyond 1024 are refused.
 */
typedef struct zero_ns_config {
  int32_t steps;
  float a;
  float b;
  float c;
  float eps;
} zero_ns_config;

/* Workspace of zero_orthogonalize for a stack of `batch` rows x cols matrices
 * (0 when there is nothing to do): 8 bytes per element of up to 2^27 and 4 per
 * element of the Gram matrices, so up to 1.6 GB unless one matrix alone is larger.
 * Errors: ZERO_EINVAL. */
zero_status zero_orthogonalize_workspace_bytes(const zero_ns_config* cfg, int64_t rows, int64_t cols, int64_t batch,
                                               int64_t* bytes);

/*
 * zero_orthogonalize — out[i] = bf16(orthogonalised in[i]) for a stack of
 * matrices.  No context: errors' text comes from zero_last_error(NULL).
 *  in         device matrices of in_dtype (zero_grad_dtype), element (r, c) of
 *             matrix i at i * in_batch_stride + r * in_row_stride + c
 *             (elements; the batch stride may be 0)
 *  out        device bf16 matrices, likewise; must not overlap `in`
 *  workspace  device scratch, 256-byte aligned, kept until the work on
 *             `stream` has completed
 * Equal calls give equal bits, and the values of a matrix's neighbours do not
 * count.  How many there are may: a smaller side of at most 128 gives the same
 * bits in any stack, for larger ones the order of the sums depends on how many
 * tiles the stack has (512 x 2048 alone, in a stack of two and of four: sums
 * over k in eight, four and two parts), and in a Muon step on the shapes that
 * share its launches.
 * Entries may have any finite size: the norm is summed so that their squares
 * stay in range.  An all-zero matrix gives zeros (with eps = 0, too); one with
 * an inf or NaN gives NaN.
 * rows, cols or batch of 0: ZERO_OK without device work.  Waits of the kernels
 * are bounded, see zero_kernel_timeouts.
 * Errors: ZERO_EINVAL (config, sizes, strides, pointers, workspace);
 * ZERO_ECUDA.
 */
zero_status zero_orthogonalize(const zero_ns_config* cfg, int64_t rows, int64_t cols, int64_t batch, const void* in,
                               int32_t in_dtype, int64_t in_row_stride, int64_t in_batch_stride, void* out,
                               int64_t out_row_stride, int64_t out_batch_stride, void* workspace,
                               int64_t workspace_bytes, void* stream);

/* Scale s of a matrix's update: 0.2 sqrt(max(rows, cols)) gives it the RMS of
 * an Adam update, so that both can share a learning rate and decay; the other
 * is sqrt(max(1, rows / cols)). */
#define ZERO_MUON_SCALE_RMS 0
#define ZERO_MUON_SCALE_ASPECT 1

/*
 *  lr, momentum, weight_decay   finite; momentum in [0, 1), decay >= 0
 *  nesterov                     1: update = g + momentum * mom; 0: mom
 *  scale                        ZERO_MUON_SCALE_*
 */
typedef struct zero_muon_config {
  float lr;
  float momentum;
  float weight_decay;
  int32_t nesterov;
  int32_t scale;
  zero_ns_config ns;
} zero_muon_config;

/* Workspace of zero_enable_muon: as zero_orthogonalize's, and 4 bytes per element
 * for the update (1.7 GB for eight 2048-wide decoder layers).  rows / cols as there.
 * Errors: ZERO_EINVAL, ZERO_ENOMEM. */
zero_status zero_muon_workspace_bytes(const zero_ctx* ctx, const zero_muon_config* cfg, const int64_t* rows,
                                      const int64_t* cols, int32_t n_params, int64_t* bytes);

/*
 * zero_enable_muon — later zero_steps update the given matrices so:
 *   g   = ((G_0 + G_1) + ... + G_{N-1}) * (1/N)   (times the clip coefficient)
 *   mom = momentum * mom + g                      (in exp_avg)
 *   u   = nesterov ? g + momentum * mom : mom
 *   w   = w * (1 - lr*weight_decay) - lr * s * orthogonalised(u)
 *   param16 = bf16(w)
 * and everything else (pads included) as before.  exp_avg_sq is not used for
 * the matrices.  Clipping (kept or not), the overflow count, capture,
 * export / import and the gathers work unchanged; zero_set_lr sets Adam's
 * rate alone.  Calling it again replaces the configuration.
 *  rows, cols  per parameter: its row-major shape, rows * cols elements; 0, 0
 *              leaves the parameter with Adam
 *  workspace   device scratch of zero_muon_workspace_bytes, 256-byte aligned,
 *              caller-owned: every later step uses it, and it must outlive the
 *              last of them on its stream, also after this call was repeated or
 *              zero_disable_muon called.  A captured step keeps the
 *              configuration and the workspace it was captured with, for as
 *              long as it is replayed
 * Errors: ZERO_EINVAL (config, shapes, workspace); ZERO_ESTATE (no buffers, a
 * step awaits post_step); ZERO_ENOTSUP (offload context); ZERO_ENOMEM.  A
 * zero_step that then fails with ZERO_ECUDA may have updated what was launched
 * before the failure.
 */
zero_status zero_enable_muon(zero_ctx* ctx, const zero_muon_config* cfg, const int64_t* rows, const int64_t* cols,
                             int32_t n_params, void* workspace, int64_t workspace_bytes);

/* All parameters back to Adam (exp_avg of the matrices then holds their
 * momentum, exp_avg_sq what it held before).  Errors: ZERO_ESTATE. */
zero_status zero_disable_muon(zero_ctx* ctx);

/* Learning rate of later Muon updates (a captured step keeps its own). */
zero_status zero_set_muon_lr(zero_ctx* ctx, float lr);

/* ---- Norm and rotation of queries and keys --------------------------------
 * Orthogonalised updates move all singular values of the query and key
 * projections at one rate, which lets attention logits grow; training with
 * them norms every head's queries and keys.  The two gains are parameters of
 * the layer's unit (vectors: Adam), and the backward pass can write their
 * gradient where the replica's flat gradient holds it.
 */

/*
 *  q_heads, k_heads  heads per token (0 allowed), head_dim 2..256 (the norm of
 *                    one element leaves its sign alone, and its gradient in
 *                    fp32 would be rounding)
 *  rotary_dim        even, 0..head_dim: the first rotary_dim elements of a head
 *                    are rotated, the rest only normed
 *  interleaved       0: element i pairs with i + rotary_dim/2; 1: 2i with 2i+1
 *  dtype             zero_grad_dtype of queries, keys and their gradients
 *  gain_dtype        zero_grad_dtype of the gains (bf16: as gathered)
 *  n_positions       rows of the rotation table
 *  eps               finite, >= 0
 */
typedef struct zero_qk_config {
  int32_t q_heads;
  int32_t k_heads;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t dtype;
  int32_t gain_dtype;
  float eps;
  int64_t n_positions;
} zero_qk_config;

/* Device heads: element d of head h of token t at t * token_stride +
 * h * head_stride + d (elements; aligned to the element size). */
typedef struct zero_heads {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} zero_heads;

/*
 * zero_qk_norm_rope — for every token t and head, with x the head's vector,
 *   y = x / sqrt(mean(x^2) + eps) * gain
 *   out = y with every pair (y1, y2) of the rotated part turned to
 *         (y1 cos - y2 sin, y2 cos + y1 sin)
 * in fp32, rounded once.  A token whose position is outside [0, n_positions)
 * is padding: its outputs are zero.  Queries and keys share one launch.
 *  q_gain, k_gain  head_dim elements of gain_dtype, or NULL: no gain
 *  table           fp32 [n_positions][rotary_dim]: rotary_dim/2 cosines, then
 *                  as many sines (NULL allowed when rotary_dim is 0)
 *  positions       int32 per token, or NULL: token t has position t
 *  q_out, k_out    may be q, k themselves (same strides), else must not
 *                  overlap them
 * tokens of 0: ZERO_OK without device work.  No context: errors' text comes
 * from zero_last_error(NULL).  Errors: ZERO_EINVAL; ZERO_ECUDA.
 */
zero_status zero_qk_norm_rope(const zero_qk_config* cfg, int64_t tokens, const zero_heads* q, const zero_heads* k,
                              const void* q_gain, const void* k_gain, const float* table, const int32_t* positions,
                              const zero_heads* q_out, const zero_heads* k_out, void* stream);

/* Workspace of zero_qk_norm_rope_backward.  Errors: ZERO_EINVAL. */
zero_status zero_qk_backward_workspace_bytes(const zero_qk_config* cfg, int64_t tokens, int64_t* bytes);

/*
 * zero_qk_norm_rope_backward — gradients of zero_qk_norm_rope's inputs from
 * those of its outputs (dq_out, dk_out), with x the forward input, xn = x *
 * rstd and h the gradient turned back by the rotation:
 *   dx = rstd * (gain h - xn mean(gain h xn)),   dgain = sum of h xn
 * over every token that is not padding (padding tokens' dx are zero, their
 * gradients are not read into any sum).  The gain sums are fp32 in a fixed
 * order: the same call gives the same bits.
 *  dq, dk            may be dq_out, dk_out or q, k themselves (same strides), else
 *                    must not overlap an input
 *  dq_gain, dk_gain  head_dim elements of dgain_dtype (zero_grad_dtype),
 *                    overwritten (zeros for 0 tokens or heads); NULL: not
 *                    wanted
 *  workspace         device scratch, 16-byte aligned
 * Errors: as zero_qk_norm_rope; ZERO_EINVAL for a small workspace.
 */
zero_status zero_qk_norm_rope_backward(const zero_qk_config* cfg, int64_t tokens, const zero_heads* dq_out,
                                       const zero_heads* dk_out, const zero_heads* q, const zero_heads* k,
                                       const void* q_gain, const void* k_gain, const float* table,
                                       const int32_t* positions, const zero_heads* dq, const zero_heads* dk,
                                       void* dq_gain, void* dk_gain, int32_t dgain_dtype, void* workspace,
                                       int64_t workspace_bytes, void* stream);

/* ---- Activations in 8 bits ---------------------------------------------------
 * What a training step keeps of its activations for the backward pass, in half
 * or a quarter of the bytes: 8-bit codes with one scale for every 32 columns of
 * a row.  A scale is the smallest power of two, from 2^-126 on, under which the
 * group's largest magnitude is at most the format's (448; 127): an element is
 * divided by it exactly and rounded once, to nearest, ties to even.  A group
 * with an inf or NaN in it reads as NaN; an entry that rounds up to 2^128 (from
 * 31/32 of it on in e4m3, above 127/128 as whole numbers) reads as inf.
 */
#define ZERO_PACK_E4M3 0  /* 4 significant bits: off by at most 2^-4 of itself or, below 2^-6 scales, 2^-10 of the scale */
#define ZERO_PACK_INT8 1  /* whole numbers: off by at most half a scale, 1/127 of the group's largest (from 2^-120 on) */

/*
 * The 8-bit form of a matrix (device memory):
 *  codes   [rows][groups * 32] bytes, 16-byte aligned; groups = ceil(cols / 32).
 *          Codes of columns that do not exist are zero
 *  scales  [rows][groups] bytes: the power of two plus 127; 255: not finite
 *  format  ZERO_PACK_*
 */
typedef struct zero_packed {
  void* codes;
  void* scales;
  int32_t format;
} zero_packed;

/*
 * zero_pack_activations — codes and scales of a matrix; zero_unpack_activations
 * — the values they stand for, rounded to dtype (exact, but for bf16
 * subnormals and 2^128: inf).
 *  cols    1..2^24; row r of the matrix begins at r * stride elements; the
 *          stride of an output is at least cols
 * rows of 0: ZERO_OK without device work.  Errors: ZERO_EINVAL; ZERO_ECUDA.
 */
zero_status zero_pack_activations(int64_t rows, int64_t cols, const void* x, int32_t dtype, int64_t x_stride,
                                  const zero_packed* packed, void* stream);
zero_status zero_unpack_activations(int64_t rows, int64_t cols, const zero_packed* packed, void* out, int32_t dtype,
                                    int64_t out_stride, void* stream);

/* ---- Layer norm ----------------------------------------------------------------
 *  cols          1..2^24
 *  center        1: layer norm; 0: the mean stays (RMS norm)
 *  dtype         zero_grad_dtype of x, y and their gradients
 *  weight_dtype  zero_grad_dtype of weight and bias (bf16: as gathered)
 *  eps           finite, >= 0
 */
typedef struct zero_norm_config {
  int64_t cols;
  int32_t center;
  int32_t dtype;
  int32_t weight_dtype;
  float eps;
} zero_norm_config;

/*
 * zero_layer_norm — for every row x
 *   mean = sum x / cols (center 0: 0),  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps)
 *   y = (x - mean) * rstd * weight + bias
 * in fp32, rounded once; a row whose squares exceed fp32's range (entries from
 * about 1e19 on) has rstd 0, and squares below it (entries under about 1e-19)
 * are lost beside any eps of an ordinary size, but leave rstd inf with eps 0.
 *  weight, bias   cols elements of weight_dtype, or NULL: none
 *  y              may be x itself (same stride), else must not overlap an input;
 *                 a stride of at least cols
 *  stats          fp32 [rows][2]: mean and rstd, which the backward pass reads;
 *                 8-byte aligned, or NULL: not wanted
 *  packed         takes the 8-bit form of x in the same pass, or NULL
 * rows of 0: ZERO_OK without device work.  Errors: ZERO_EINVAL; ZERO_ECUDA.
 */
zero_status zero_layer_norm(const zero_norm_config* cfg, int64_t rows, const void* x, int64_t x_stride,
                            const void* weight, const void* bias, void* y, int64_t y_stride, float* stats,
                            const zero_packed* packed, void* stream);

/* Workspace of zero_layer_norm_backward.  Errors: ZERO_EINVAL. */
zero_status zero_layer_norm_backward_workspace_bytes(const zero_norm_config* cfg, int64_t rows, int64_t* bytes);

/*
 * zero_layer_norm_backward — with xn = (x - mean) * rstd, g = dy * weight:
 *   dx = rstd * (g - sum g / cols - xn * sum (g xn) / cols)   (center 0: without sum g)
 *   dweight = sum over the rows of dy xn,  dbias = sum over the rows of dy
 * The column sums are fp32 in an order that the sizes, types, strides and
 * alignments fix: the same call gives the same bits.
 *  x, packed         the forward input, or (x NULL) its 8-bit form; the entries
 *                    it stands for take the input's place, the statistics stay
 *  stats             as zero_layer_norm wrote them
 *  dx                may be dy or x itself (same stride), else must not overlap
 *                    an input; a stride of at least cols
 *  dweight, dbias    cols elements of dgrad_dtype (zero_grad_dtype), overwritten
 *                    (zeros for 0 rows); NULL: not wanted
 *  workspace         device scratch, 16-byte aligned (not read where neither of
 *                    the two is wanted)
 * Errors: as zero_layer_norm; ZERO_EINVAL for a small workspace.
 */
zero_status zero_layer_norm_backward(const zero_norm_config* cfg, int64_t rows, const void* dy, int64_t dy_stride,
                                     const void* x, int64_t x_stride, const zero_packed* packed, const void* weight,
                                     const float* stats, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                     int32_t dgrad_dtype, void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Embedding -----------------------------------------------------------------
 *  rows      of the table, 0..2^30
 *  dim       1..2^24
 *  dtype     zero_grad_dtype of the table and of the looked up rows (forward),
 *            of their gradient (backward)
 *  id_bytes  4 or 8: int32 or int64 ids
 *  scale     finite factor of the looked up rows
 */
typedef struct zero_embedding_config {
  int64_t rows;
  int64_t dim;
  int32_t dtype;
  int32_t id_bytes;
  float scale;
} zero_embedding_config;

/*
 * zero_embedding — out[t] = scale * table[ids[t]], rounded once; zeros where the
 * id is outside [0, rows) (padding).
 *  tokens   0..2^30 (0: ZERO_OK without device work)
 *  table, out   rows at multiples of their stride (elements); that of out is at
 *               least dim
 * Errors: ZERO_EINVAL; ZERO_ECUDA.
 */
zero_status zero_embedding(const zero_embedding_config* cfg, int64_t tokens, const void* ids, const void* table,
                           int64_t table_stride, void* out, int64_t out_stride, void* stream);

/* Workspace of zero_embedding_backward.  Errors: ZERO_EINVAL. */
zero_status zero_embedding_backward_workspace_bytes(const zero_embedding_config* cfg, int64_t tokens, int64_t* bytes);

/*
 * zero_embedding_backward — dtable[v] = scale * sum of dout[t] over the tokens t
 * with ids[t] = v.  The tokens are sorted by row, the sums fp32 in an order that
 * the ids fix: the same call gives the same bits.
 *  tokens      0..2^30, and at most 2^50 over the rows rounded up to a power of
 *              two: every 1024 rows (from 2^17 rows on) read all ids
 *  dtable      dtable_dtype (zero_grad_dtype), must not overlap dout or ids; a
 *              stride of at least dim
 *  accumulate  0: every row is written (zeros without tokens); 1: the sums are
 *              added to what is there, rows without tokens stay as they are
 *  workspace   device scratch, 16-byte aligned
 * Errors: as zero_embedding; ZERO_EINVAL for a small workspace.
 */
zero_status zero_embedding_backward(const zero_embedding_config* cfg, int64_t tokens, const void* ids, const void* dout,
                                    int64_t dout_stride, void* dtable, int32_t dtable_dtype, int64_t dtable_stride,
                                    int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * zero_kernel_timeouts — how many bounded waits of the Newton-Schulz
 * products (zero_orthogonalize, the Muon step) and of the tile-staged step
 * kernels (used for N = 1..4 or N >= 11 bf16 and N >= 7 fp32 replicas when a
 * launch covers at least 2^23 elements) gave up on the current device since
 * the library was loaded.  A wait gives up only if a
 * bulk copy or a product never arrives; the CTA then leaves the rest of its
 * tiles unchanged, so a count that grew means that a step or an
 * orthogonalisation is incomplete (its call has returned ZERO_OK before).
 * Reads device counters: synchronizes with the device.  ctx may be NULL.
 */
zero_status zero_kernel_timeouts(const zero_ctx* ctx, uint32_t* count);

/*
 * zero_debug_inject — test hook for the bounded waits above (the pages have
 * no counterpart).  what = ZERO_INJECT_MISSING_COPY arms it for the next
 * zero_step: if that step's first launch uses a tile-staged kernel, the
 * kernel announces the bytes of the launch's first tile to its mbarrier but
 * issues no copy for it, so that one wait runs out after about a second;
 * the CTA then counts a timeout (zero_kernel_timeouts), waits for the copies
 * it did issue and leaves, and the elements of its tiles stay un-updated.
 * Nothing faults: the device stays usable.  what = 0 disarms.  The hook is
 * consumed by the next vector launch whichever kernel it uses.
 * Errors: ZERO_EINVAL (NULL ctx, unknown value).
 */
#define ZERO_INJECT_MISSING_COPY 1
/*
 * what = ZERO_INJECT_SHORT_BOUNDS: the next zero_step tells its kernels that
 * the state arrays end 8 elements before they really do (the buffers keep
 * their full size, so no access can leave them).  In a debug build the index
 * checks then refuse the last 8 elements (counted, not updated); in a release
 * build the checks do not exist and the step is the normal one.
 */
#define ZERO_INJECT_SHORT_BOUNDS 2
zero_status zero_debug_inject(zero_ctx* ctx, int32_t what);

/*
 * zero_debug_check_failures — in a debug build of the library (compiled with
 * -DZFS_DEBUG_CHECKS: every kernel index is checked before the access it
 * guards; a failed check is counted and the access skipped, never trapped),
 * the number of failed checks on the current device since the library was
 * loaded.  Synchronizes with the device.  The pages have no counterpart.
 * Errors: ZERO_EINVAL (NULL); ZERO_ENOTSUP in a release build (*count = 0);
 * ZERO_ECUDA.
 */
zero_status zero_debug_check_failures(uint32_t* count);

/* Number of steps taken (t).  In capturable mode it is read from the device
 * (synchronizing), and ZERO_ESTATE reports steps skipped past max_steps. */
zero_status zero_step_count(const zero_ctx* ctx, int64_t* t);

/*
 * Number of kernels the last zero_step / zero_gather_weights / zero_gather_units call on this
 * context enqueued (0 when it had nothing to do).  Host bookkeeping only.
 */
zero_status zero_last_launches(const zero_ctx* ctx, int32_t* launches);

/* Set the learning rate used by later steps (a scheduler's lr update).  A
 * step already captured into a CUDA graph keeps the lr (and the AdamW factor
 * 1 - lr*wd) it was captured with: capture it again after a change. */
zero_status zero_set_lr(zero_ctx* ctx, float lr);

/* Release the context's host metadata.  Device buffers stay the caller's. */
zero_status zero_destroy(zero_ctx* ctx);

/*
 * Text of the last error on `ctx`; with ctx == NULL, the last error of a
 * failed zero_plan / zero_make_master on the calling thread.  The string is
 * owned by the library and valid until the next call on the same context
 * (or thread).
 */
const char* zero_last_error(const zero_ctx* ctx);

/* Constant name of a status code. */
const char* zero_status_string(zero_status status);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_FLATSTEP_H */
