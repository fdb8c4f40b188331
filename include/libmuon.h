/*
 * libmuon -- the Muon optimizer step on one AMD Instinct MI355X (gfx950).
 *
 * One call of muon_step() performs, for every 2-D hidden weight (or every
 * independent row block of one), the momentum update, Frobenius
 * normalization, the Newton-Schulz orthogonalization and the scaled,
 * decoupled-weight-decay update; every other parameter takes the elementwise
 * AdamW fallback.  All work is hand-written HIP for gfx950.
 *
 * Sources (web pages, cited by title and section):
 *   [Blog]      "Muon Optimizer and the Distributed Implementation"
 *   [Moonlight] the Kimi/Moonlight summary page ("...Muon优化器可替代 AdamW..."),
 *               sections "权重衰减机制", "参数更新尺度调整:一致的更新 RMS", "代码"
 *   [DeepSpeed] "DeepSpeed 集成 Muon 优化器实战..." (NS_METHODS, Gram variant)
 *   [MindSpeed] the MindSpeed "Muon 优化器" document (QKV split)
 *
 * Conventions shared by every entry point
 *   - Device pointers are HIP device addresses (e.g. torch tensors'
 *     data_ptr()).  The caller owns every buffer and the stream; the library
 *     never allocates device memory.  Scratch memory is the caller-provided
 *     workspace whose size the *_workspace_bytes queries return.
 *   - Matrices are row-major with a leading dimension equal to their column
 *     count unless an ld argument says otherwise.
 *   - Calls only enqueue work on the given stream (a hipStream_t passed as
 *     void*, NULL = the default stream); they never synchronize the host.
 *   - Every argument is validated on the host before the first launch; on any
 *     error nothing is enqueued and a negative muon_status is returned.
 *   - Non-finite values in the data are not checked; they propagate.
 *   - A workspace may not be used by two calls that overlap in time.
 */
#ifndef LIBMUON_H
#define LIBMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_E_ARG = -1,       /* null/misaligned pointer, bad count, non-finite hparam */
  MUON_E_SHAPE = -2,     /* negative size, split_rows not dividing rows, ... */
  MUON_E_DTYPE = -3,     /* unknown dtype code */
  MUON_E_METHOD = -4,    /* unknown ns_method */
  MUON_E_WORKSPACE = -5, /* workspace null or smaller than required */
  MUON_E_HIP = -6,       /* a HIP runtime call or kernel launch failed */
  MUON_E_PLAN = -7,      /* plan and call disagree (table size, ...) */
  MUON_E_CAPACITY = -8   /* output array too small (query calls) */
} muon_status;

/* [DeepSpeed] NS_METHODS = {standard, gram}: the standard iteration on the
 * m x n unit, or the Gram variant, which iterates on the square R = X X^T
 * (m = min, n = max of the unit's sides).  The Gram chain runs in fp16 with
 * R scaled by a power of two only where that stays within the bf16
 * tolerance on the workload gradients, m >= 512 and n >= 3m.  An explicit
 * MUON_NS_GRAM outside that region is served in a precision that meets the
 * tolerance of the requested compute dtype: with bf16 the unit's Gram
 * iteration runs in fp32 (the bucket reports compute dtype MUON_F32); with fp32 the unit
 * runs the standard iteration (the bucket reports MUON_NS_STANDARD), since
 * an fp32 Gram chain there exceeds the fp32 tolerance.  MUON_NS_AUTO picks
 * Gram exactly inside the region, where it also does less work (executed
 * cost with symmetric products: standard steps (3 m^2 n + m^3), Gram
 * 3 m^2 n + (6 steps - 5) m^3, so Gram is cheaper for n/m > 5/3), and the
 * standard method elsewhere.  MUON_NS_GRAM_RESTART is an extension (the
 * pages describe no restart): the Gram chain with one restart after
 * ceil(steps / 2) steps (steps >= 2), which forms X_r = Q X_0 explicitly,
 * recomputes R = X_r X_r^T from it and continues with Q = I, so the fp16
 * chain's rounding restarts from the rectangular iterate.  A 16-bit unit
 * with m >= 256 runs it in fp16 at any aspect ratio (at most 0.92e-2 where
 * the plain fp16 chain reaches 1.9-17e-2 on small and square shapes; the
 * bucket reports MUON_NS_GRAM_RESTART); a smaller or fp32 unit resolves as
 * for MUON_NS_GRAM.  It costs one more n x m product and one more
 * m x m x n Gram product per unit.
 * Plans report the method and compute dtype of every bucket. */
typedef enum {
  MUON_NS_STANDARD = 0,
  MUON_NS_GRAM = 1,
  MUON_NS_AUTO = 2,
  MUON_NS_GRAM_RESTART = 3
} muon_ns_method;

/* Storage dtype of parameters and gradients.  Momentum and AdamW moments are
 * fp32, but for the moments of MUON_KIND_ADAMW8. */
typedef enum { MUON_F32 = 0, MUON_BF16 = 1 } muon_dtype;

/* [Moonlight] "代码": parameters tagged use_muon take the Muon rule, the rest
 * (embeddings, heads, norms, biases) take the AdamW backup.  An extension:
 * MUON_KIND_ADAMW8 is the AdamW backup with its two moments kept in 8 bits
 * (see muon_adamw8_state_bytes); 2 is not a kind. */
typedef enum { MUON_KIND_MUON = 0, MUON_KIND_ADAMW = 1, MUON_KIND_ADAMW8 = 3 } muon_kind;

/* One row of the shape table (plan time; no pointers).
 *   rows, cols  the 2-D view of the parameter (callers flatten ndim > 2 as
 *               [size(0), -1], as the [Moonlight] code does; vectors 1 x len).
 *   split_rows  0: the whole matrix is one unit.  h > 0: rows must be a
 *               multiple of h and each block of h consecutive rows is
 *               orthogonalized on its own ([MindSpeed] QKV split; per-head
 *               split).  Muon kind only.
 *   scale_dim   0: the update scale is rms_scale*sqrt(max(unit rows, cols));
 *               d > 0: rms_scale*sqrt(d) ([Moonlight] "参数更新尺度调整"). */
typedef struct {
  int32_t kind;   /* muon_kind */
  int32_t dtype;  /* muon_dtype of param and grad */
  int64_t rows;
  int64_t cols;
  int64_t split_rows;
  int64_t scale_dim;
} muon_param_shape;

/* Device pointers of one parameter for one step (same order as the table).
 *   param     rows x cols, dtype; updated in place.
 *   grad      rows x cols, dtype; read only.
 *   momentum  rows x cols fp32 (Muon kind); updated in place.
 *   exp_avg, exp_avg_sq  rows x cols fp32 (AdamW kind); updated in place.
 *             MUON_KIND_ADAMW8: device buffers of muon_adamw8_state_bytes
 *             bytes each, 4-byte aligned (cast to float*).
 *   update_out  optional (may be NULL), Muon kind: rows x cols fp32 receives
 *             the orthogonalized update O of every unit (before scaling).
 * Alignment: param/grad to their element size, fp32 buffers to 4 bytes. */
typedef struct {
  void* param;
  const void* grad;
  float* momentum;
  float* exp_avg;
  float* exp_avg_sq;
  float* update_out;
} muon_param_ptrs;

/* Scale of the orthogonalized update O in W <- W (1 - lr wd) - lr scale O,
 * per unit, with d_out x d_in the unit's shape in parameter layout (rows x
 * cols) and D = scale_dim if set, else max(d_out, d_in):
 *   MUON_SCALE_MOONLIGHT  rms_scale * sqrt(D)            ([Moonlight]
 *                         "参数更新尺度调整": matched update RMS, 0.2)
 *   MUON_SCALE_SPECTRAL   sqrt(d_out / d_in)             ([Blog] "Variation
 *                         of Muon Optimizer": dualizing under the RMS->RMS
 *                         norm, the muP form)
 *   MUON_SCALE_UNIT_RMS   sqrt(D)                        ([Blog] DeepSeek-V4
 *                         listing, "Rescale update RMS", with gamma below)
 * each multiplied by extra_scale (the listing's update rescaling factor
 * gamma; [MindSpeed] --muon-extra-scale-factor).  MindSpeed names the modes
 * spectral / unit_rms_norm / shape_scaling without defining them; they are
 * read as SPECTRAL / UNIT_RMS / MOONLIGHT. */
typedef enum {
  MUON_SCALE_MOONLIGHT = 0,
  MUON_SCALE_SPECTRAL = 1,
  MUON_SCALE_UNIT_RMS = 2
} muon_scale_mode;

/* Hyperparameters of one step.
 *   lr, momentum, weight_decay, nesterov, ns_steps: the Muon rule
 *     ([Blog] "Formulation of Muon Optimizer"; [Moonlight] "权重衰减机制").
 *   coeffs: host array of ns_steps*3 floats (a_k, b_k, c_k) or NULL for the
 *     quintic (3.4445, -4.7750, 2.0315) at every step ([Blog] "Newton-Schulz
 *     Iteration").
 *   rms_scale: 0.2 in [Moonlight]; with the default scale mode the update
 *     is W <- W (1 - lr wd) - lr rms_scale sqrt(max(A,B)) O.
 *   scale_mode: muon_scale_mode (0 = MOONLIGHT).
 *   extra_scale: multiplier of the scale; 0 is read as 1 (so a zeroed struct
 *     keeps the default rule).  Must be finite and >= 0.
 *   adam_*: the AdamW backup of the [Moonlight] code; adam_step is t >= 1
 *     (already incremented): W <- W (1 - lr wd) - lr sqrt(1-b2^t)/(1-b1^t) *
 *     m / (eps + sqrt(v)). */
typedef struct {
  float lr;
  float momentum;
  float weight_decay;
  int32_t nesterov;
  int32_t ns_steps;
  const float* coeffs;
  float rms_scale;
  float adam_lr;
  float adam_beta1;
  float adam_beta2;
  float adam_eps;
  float adam_weight_decay;
  int64_t adam_step;
  int32_t scale_mode;
  float extra_scale;
} muon_hparams;

/* The moments of a MUON_KIND_ADAMW8 parameter, in 8 bits each.  A step computes
 * in fp32, each operation rounded by itself,
 *   m <- m + (1-b1) (g - m);  v <- v + (1-b2) (g g - v);
 *   W <- W (1 - lr wd) - lr sqrt(1-b2^t)/(1-b1^t) m / (eps + sqrt(v))
 * with m and v as they are, and then rounds them to what is kept:
 * Blocks of 256 elements in a row of the parameter's memory share an offset o.
 * With u(x) the bits of the float x >= 0,
 *   o = max(0, ceil(max u(x) / 2^20) - K),  K = 127 for |m|, 255 for v,
 * an element's code k stands for the float of bits (k + o) 2^20, and for zero
 * where k = 0; the code of m has its sign in bit 7.  That is 3 bits of
 * mantissa and 15.9 (m) or 31.9 (v) powers of two below the block's largest.
 *   k = floor((u(x) + 16 r) / 2^20) - o,  r uniform in 0 .. 65535:
 * a value is rounded up or down with the probabilities that keep its mean
 * (nearest rounding would hold v where it is: a step takes at most 1-b2 off
 * it).  Under the smallest code lo (o + 1 as bits), m gets lo where
 * |m| > lo (r + 1/2) / 65536 and else 0, and v > 0 gets lo.  NaN and infinity
 * are kept, and lower the rest of their block to 0 or lo; finite values of at
 * least 1.875 2^127 may become infinite.
 * r comes from the step's number t and the element's index i: with
 *   mix(x): x ^= x >> 16; x *= 0x6a09e667; x ^= x >> 15; x *= 0xbb67ae85;
 *           x ^= x >> 16     (all modulo 2^32)
 *   key = mix(lo32(t) ^ mix(hi32(t))),  q = i / 4,
 *   h = mix(lo32(q) ^ (hi32(q) * 0x9e3779b1) ^ key) rotated right by 8 (i % 4),
 * r is the low half of h for m and the high half for v.  So a step's result
 * follows from its inputs, whatever else the step updates.
 * Storage: the codes of ceil(numel / 256) whole blocks, then a 16-bit offset
 * per block, then up to the next multiple of 16 bytes.  All zero bytes are
 * zero moments (a new parameter's).  Codes behind the last element are left as
 * they are.  The size is a multiple of 16 bytes, so buffers that follow each
 * other without gaps stay aligned.
 * adam_beta1 and adam_beta2 are in [0, 1) for such parameters.
 *
 * muon_adamw8_state_bytes: bytes of one moment (host only).
 * muon_adamw8_pack: fp32 values x to a moment's buffer, rounded as in step
 *   `step` (codes behind the last element become 0, bytes behind the offsets
 *   are left).  MUON_ADAMW8_SECOND takes |x|.
 * muon_adamw8_unpack: the values that a buffer stands for.
 * Errors: MUON_E_METHOD (unknown moment), MUON_E_SHAPE (numel negative or above
 * 2^40), MUON_E_ARG (a pointer null or not 4-byte aligned), MUON_E_HIP. */
typedef enum { MUON_ADAMW8_FIRST = 0, MUON_ADAMW8_SECOND = 1 } muon_adamw8_moment;
muon_status muon_adamw8_state_bytes(int64_t numel, size_t* bytes);
muon_status muon_adamw8_pack(const float* x, int64_t numel, int32_t moment, int64_t step, void* state, void* stream);
muon_status muon_adamw8_unpack(const void* state, int64_t numel, int32_t moment, float* x, void* stream);

/* Plan options.
 *   ns_method  muon_ns_method.
 *   ns_dtype   -1: Newton-Schulz computes in the parameter dtype (bf16 MFMA
 *              for bf16 parameters, fp32 MFMA for fp32 ones); MUON_F32 or
 *              MUON_BF16 forces one. */
typedef struct {
  int32_t ns_method;
  int32_t ns_dtype;
} muon_plan_options;

typedef struct muon_plan muon_plan;

/* Build an immutable plan from a shape table of n rows (table: host array
 * owned by the caller, read only during the call): units (one per matrix
 * or row block) grouped into buckets of equal (m, n, tall, parameter
 * dtype, compute dtype, method), m = min and n = max of the unit's sides.
 * Which parameters take the Muon rule and which the AdamW backup follows
 * [Moonlight] "代码" (use_muon; Muon only for 2-D weights); a split
 * parameter's row blocks are orthogonalized independently, as the fused QKV
 * weight is in [MindSpeed] "TP 兼容适配" (Q, K, V blocks) and per attention
 * head in [DeepSpeed] (Muon Split); a tall unit is processed as its
 * transpose ([Blog] "Sign of a Matrix": msign(G) = G (G^T G)^(-1/2)).
 * Buckets are numbered by first appearance; units keep table order.  Host
 * only (no HIP call).  opts may be NULL (standard method, compute dtype of
 * the parameters).  *out receives a heap object to release with
 * muon_plan_destroy.  Errors: MUON_E_ARG (null out, n < 0, unknown kind),
 * MUON_E_DTYPE, MUON_E_METHOD, MUON_E_SHAPE (negative size, side > 2^30,
 * split_rows not dividing rows or set on an AdamW row, a unit whose
 * working copy reaches 2^31 bytes, a MUON_KIND_ADAMW8 row of more than 2^40
 * elements); on error *out is NULL. */
muon_status muon_plan_create(const muon_param_shape* table, int32_t n,
                             const muon_plan_options* opts, muon_plan** out);
void muon_plan_destroy(muon_plan* plan);

/* Bytes of device workspace muon_step needs with this plan (host only).
 * The workspace holds, per bucket chunk, the working copies of the
 * Newton-Schulz iteration ([Blog] "Newton-Schulz Iteration": X and its
 * transpose-side products A = X X^T and P = aI + bA + cA^2, or the Gram
 * variant's R, P and Q of [DeepSpeed]), the per-unit norms and the device
 * descriptor tables.  0 for a plan without units or AdamW parameters.
 * Errors: MUON_E_ARG (null plan or bytes). */
muon_status muon_plan_workspace_bytes(const muon_plan* plan, size_t* bytes);

/* Bit-exact view of the plan (host only).  Buckets: 8 int32 per bucket
 * (m, n, tall, param dtype, compute dtype, method, first unit, unit count);
 * units, listed bucket by bucket: 6 int64 per unit (param, row0, rows, cols,
 * tall, scale_dim as resolved).  *len receives the number of values needed;
 * with out == NULL and cap == 0 this is a size query (MUON_OK), otherwise a
 * cap below it returns MUON_E_CAPACITY and writes nothing. */
muon_status muon_plan_buckets(const muon_plan* plan, int32_t* out, size_t cap, size_t* len);
muon_status muon_plan_units(const muon_plan* plan, int64_t* out, size_t cap, size_t* len);

/* One optimizer step for every parameter of the plan's table (n must equal
 * the table size; ptrs: host array of n entries in table order, read only
 * during the call; hp: host struct, read only during the call).
 * Per Muon unit ([Blog] "Formulation of Muon Optimizer" and "Newton-Schulz
 * Iteration"; [Moonlight] "权重衰减机制", "参数更新尺度调整" and "代码"):
 *   M <- mu M + G;  U = G + mu M (nesterov) or M;  X0 = U / ||U||_F;
 *   X <- a_k X + (b_k A + c_k A^2) X, A = X X^T, k = 0 .. ns_steps-1
 *     (or the Gram variant of [DeepSpeed]);
 *   W <- W (1 - lr wd) - lr scale O, scale per muon_scale_mode;
 * a unit whose U is zero gets O = 0 (its weight only decays).  Per AdamW
 * parameter: the AdamW backup of [Moonlight] "代码" (see muon_hparams).
 * param, momentum, exp_avg, exp_avg_sq are updated in place and update_out
 * written; grad is read only.  workspace: device memory of at least
 * muon_plan_workspace_bytes bytes, owned by the caller; its contents need
 * not be initialized and are scratch between calls.  The per-unit
 * descriptors reach the workspace through the arguments of small kernel
 * launches (3 KiB each), not through a host-to-device copy, so the call
 * only enqueues work on stream (a hipStream_t, NULL = default stream) and
 * returns without waiting for the GPU.  Errors, all before the first
 * launch: MUON_E_PLAN (n
 * differs from the table), MUON_E_ARG (null plan, hp or ptrs; a required
 * pointer null or misaligned; a non-finite or out-of-range hparam),
 * MUON_E_WORKSPACE; MUON_E_HIP if a HIP call fails. */
muon_status muon_step(const muon_plan* plan, const muon_param_ptrs* ptrs, int32_t n,
                      const muon_hparams* hp, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Newton-Schulz orthogonalization of one matrix X (device memory, rows x
 * cols, leading dimension ld >= cols elements, dtype MUON_F32 or MUON_BF16),
 * in place: X <- NS_steps(X / ||X||_F) ([Blog] "Newton-Schulz Iteration":
 * X <- a_k X + (b_k A + c_k A^2) X with A = X X^T), a tall X being processed
 * as its transpose ([Blog] "Sign of a Matrix"); method standard, Gram
 * ([DeepSpeed]; resolved as described above), auto, or the restarted Gram
 * chain (an extension, resolved as described above).
 * coeffs: host array of steps x 3 floats as in muon_hparams, or NULL.  A
 * zero matrix stays zero.  workspace: device memory of at least
 * ns_orthogonalize_workspace_bytes bytes, owned by the caller, contents
 * need not be initialized.  Enqueues on stream and returns.  Errors, before
 * any launch: MUON_E_DTYPE, MUON_E_METHOD, MUON_E_SHAPE (negative size,
 * ld < cols, a side above 2^30 or a working copy of 2^31 bytes or more),
 * MUON_E_ARG (X null or misaligned, steps out of [1, 64], a non-finite
 * coefficient), MUON_E_WORKSPACE; MUON_E_HIP if a launch fails. */
muon_status ns_orthogonalize(void* X, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                             int32_t steps, const float* coeffs, int32_t method,
                             void* workspace, size_t workspace_bytes, void* stream);
muon_status ns_orthogonalize_workspace_bytes(int64_t rows, int64_t cols, int32_t dtype,
                                             int32_t method, size_t* bytes);

/* ns_orthogonalize without a workspace argument, for callers that cannot
 * allocate device memory (code under stream capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The arguments of ns_orthogonalize less
 * the workspace; the same result and errors as
 * ns_orthogonalize, with the same kernels; the scratch memory is a device
 * array of MUON_NOALLOC_SCRATCH_BYTES inside the library, one per GPU the
 * library is loaded on, held until the process ends.  The call allocates
 * nothing: no hipMalloc / hipFree, no host staging.  Matrices whose
 * ns_orthogonalize_workspace_bytes exceed MUON_NOALLOC_SCRATCH_BYTES (e.g. a
 * bf16 2048 x 4096 fits, a 4096 x 4096 does not) return MUON_E_WORKSPACE
 * before any launch.  Every call on one GPU uses that GPU's one array: calls
 * that overlap in time on the same GPU (two streams, two threads) race and
 * must be serialized by the caller.  The array's contents after a call are
 * unspecified; nothing needs to be zero before one.  MUON_E_HIP if the
 * array's device address cannot be obtained. */
#define MUON_NOALLOC_SCRATCH_BYTES (64u << 20)
muon_status ns_orthogonalize_noalloc(void* X, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                                     int32_t steps, const float* coeffs, int32_t method, void* stream);

/* Optional per-kernel timing, for benchmarks.  While enabled (process-wide),
 * every kernel launch of the library is bracketed by two HIP events recorded
 * on the launch's stream, tagged with the kernel family and the algorithmic
 * FLOPs / HBM bytes of that launch:
 *   flops  Newton-Schulz contractions: 2*m*m*n (X X^T and P X) or 2*m^3
 *          (A A and the Gram m x m products) per unit, counted as dense
 *          products even where symmetry halves the executed work;
 *   bytes  elementwise kernels: bytes each element must move (momentum:
 *          G + M read + M write + U write; AdamW: W r/w, G, m r/w, v r/w).
 * muon_timing_collect waits for the recorded events, writes one entry per
 * family into out (up to cap), sets *n to the number of families seen, and
 * clears the records. */
typedef struct {
  char name[32];
  int64_t launches;
  double total_ms;
  double flops;
  double bytes;
} muon_kernel_timing;

muon_status muon_timing_enable(int32_t enable);
muon_status muon_timing_collect(muon_kernel_timing* out, int32_t cap, int32_t* n);

/* Measurement aids for benchmarks; not part of the optimizer step.  Both
 * only enqueue on stream (a hipStream_t, null = default stream) and return.
 * muon_probe_mfma: the device's sustained bf16 matrix-core rate.  Launches
 *   `workgroups` workgroups of 4 waves; each wave runs `iters` rounds of 8
 *   independent v_mfma_f32_32x32x16_bf16 from registers, and each workgroup
 *   writes one float to sink (device memory, `workgroups` floats, owned by
 *   the caller).  *flops (host) receives the FLOPs of the launch
 *   (workgroups * 4 * iters * 8 * 32768).  MUON_E_ARG if a count is not
 *   positive or a pointer is null; MUON_E_HIP if the launch fails.
 * muon_probe_copy: the device's streaming copy rate.  Copies `bytes` from
 *   src to dst (device memory, non-overlapping, owned by the caller) with
 *   16-byte non-temporal loads and stores, one contiguous 16 KiB block per
 *   workgroup; 2 * bytes move through HBM.
 *   MUON_E_ARG if bytes is 0 or not a multiple of 16, or a pointer is null
 *   or not 16-byte aligned; MUON_E_HIP if the launch fails. */
muon_status muon_probe_mfma(int32_t workgroups, int32_t iters, float* sink, double* flops, void* stream);
muon_status muon_probe_copy(const void* src, void* dst, size_t bytes, void* stream);
/* muon_probe_copy_lds: the same copy through the Newton-Schulz GEMMs' load
 *   path (global -> LDS with buffer_load_dwordx4 ... lds at the default cache
 *   policy, then LDS -> global with ordinary 16-byte stores), one 16 KiB
 *   block per workgroup; calibrates memory counters for those loads.  Same
 *   arguments and errors as muon_probe_copy. */
muon_status muon_probe_copy_lds(const void* src, void* dst, size_t bytes, void* stream);

/* Newton-Schulz coefficient schedules: writes steps x 3 floats (a_k, b_k,
 * c_k) to out (capacity cap floats) for muon_hparams.coeffs.
 *   MUON_COEFF_QUINTIC  (3.4445, -4.7750, 2.0315) at every step ([Blog]
 *                       "Newton-Schulz Iteration"; [MindSpeed]
 *                       --muon-coefficient-type quintic).
 *   MUON_COEFF_HYBRID   the quintic for steps-2 steps, then two refining
 *                       steps ([Blog] DeepSeek-V4 listing: HybridNewtonSchulz,
 *                       ten steps, eight with the quintic and two with an
 *                       improved Newton iteration that brings the singular
 *                       values closer to 1).  The refined coefficients are not
 *                       printed; the reading taken is (15/8, -5/4, 3/8), the
 *                       odd quintic with p(1) = 1, p'(1) = p''(1) = 0 (the
 *                       second-order expansion of [Blog] "Sign of a Matrix").
 *                       steps >= 2.
 * Errors: MUON_E_ARG (unknown kind, steps out of [1, 64], hybrid with
 * steps < 2, null out), MUON_E_CAPACITY (cap < 3 steps). */
typedef enum { MUON_COEFF_QUINTIC = 0, MUON_COEFF_HYBRID = 1 } muon_coeff_kind;
muon_status muon_ns_coefficients(int32_t kind, int32_t steps, float* out, size_t cap);

/* ---------------------------------------------------------------------------
 * The operators around the step: what makes the gradients muon_step reads.
 *
 * Norms give the gradients of a table's AdamW vectors (layer norm weights and
 * biases, RMS norm weights); the linear layer on 8-bit rows gives those of
 * its Muon matrices from activations that were kept in 8 bits.  They follow
 * the conventions above; in addition
 *   - matrices take a leading dimension (elements between rows) of at least
 *     their column count; only the rows x cols values are read or written
 *     unless a comment says otherwise;
 *   - dtype codes are muon_dtype; sums, statistics and products are held in
 *     32 bits and rounded once on output;
 *   - an output must not overlap an input, except where said;
 *   - results do not depend on the stream, on other calls or on timing: sums
 *     are joined in a fixed order.
 * ------------------------------------------------------------------------- */

/* 8-bit rows: a rows x cols matrix held as int8 q (leading dimension ldq) and
 * one fp32 scale per row, standing for q[i][j] * scale[i].
 *   scale[i] = 2^e, e the smallest integer with max_j |x[i][j]| <= 127 * 2^e,
 *              not below -126 (an all-zero row has 2^-126);
 *   q[i][j]  = x[i][j] / scale[i] rounded to nearest even, in [-127, 127]
 *              (in [-63, 63] where e is 122, its largest value, so that every
 *              q * scale is finite).
 * A row that holds a NaN or an infinity gets scale NaN and q = 0, so whatever
 * is computed from it is NaN.  A power of two costs up to one of the 8 bits
 * against max / 127 and makes q * scale exact in bf16, so restoring a row and
 * feeding it to bf16 matrix instructions rounds nothing.
 * Storage: q is 16-byte aligned, ldq is a multiple of 16, every row's ldq
 * bytes belong to the buffer, and the bytes from cols up to the next
 * multiple of 16 are zero.  muon_rows8_quantize and muon_norm_forward write
 * those zeros; the bytes behind them are left as they are. */
muon_status muon_rows8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t dtype,
                                int8_t* q, int64_t ldq, float* scale, void* stream);
/* y[i][j] = q[i][j] * scale[i] (y may be bf16 or fp32; exact for the scales
 * muon_rows8_quantize writes, apart from bf16's range at its far ends).
 * Errors of both: MUON_E_DTYPE; MUON_E_SHAPE (a size negative, rows above
 * 2^30, cols above 2^27, a leading dimension below cols or above 2^40, ldq not a multiple of 16);
 * MUON_E_ARG (a pointer null or not aligned: x and y to their element, q to
 * 16 bytes, scale to 4); MUON_E_HIP. */
muon_status muon_rows8_dequantize(const int8_t* q, int64_t ldq, const float* scale, int64_t rows, int64_t cols,
                                  void* y, int64_t ldy, int32_t dtype, void* stream);

/* Row norms.  Per row x of cols values (all rows independent):
 *   mu = mean(x) (MUON_NORM_LAYER) or 0 (MUON_NORM_RMS)
 *   r  = 1 / sqrt(mean((x - mu)^2) + eps),  h = (x - mu) r
 *   y  = h gamma + beta
 * The squares are summed in fp32: a row whose sum of (x - mu)^2 passes 2^128
 * gets r = 0. */
typedef enum { MUON_NORM_LAYER = 0, MUON_NORM_RMS = 1 } muon_norm_kind;

/* x: rows x cols, dtype.  gamma, beta: cols values of vec_dtype; beta may be
 * NULL.  Outputs, each optional, at least one given:
 *   y (dtype, ldy); may be x itself (with ldy == ldx)
 *   q, ldq, scale: y, before any rounding to dtype, as 8-bit rows (both or neither)
 *   mean, rstd: rows fp32 values of mu and r, for the backward pass (mean must
 *     be NULL for MUON_NORM_RMS).
 * With rows == 0 or cols == 0 nothing is read or written: a row without values
 * has no statistics, and its 8-bit form needs no scale (see
 * muon_linear8_forward; muon_rows8_quantize writes 2^-126).
 * Errors: MUON_E_METHOD (unknown kind), MUON_E_DTYPE, MUON_E_SHAPE (as for
 * muon_rows8_quantize), MUON_E_ARG (a required pointer null, any pointer
 * misaligned, eps negative or not finite, no output), MUON_E_HIP. */
muon_status muon_norm_forward(int32_t kind, const void* x, int64_t rows, int64_t cols, int64_t ldx, int32_t dtype,
                              const void* gamma, const void* beta, int32_t vec_dtype, float eps, void* y,
                              int64_t ldy, int8_t* q, int64_t ldq, float* scale, float* mean, float* rstd,
                              void* stream);

/* Gradients of muon_norm_forward, with g = dy gamma and the saved mean, rstd:
 *   dx     = r (g - mean(g) - h mean(g h))   (MUON_NORM_RMS: without mean(g))
 *   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
 * dy, x, dx: rows x cols, dtype; dx may be dy itself (with lddx == lddy).
 * dgamma, dbeta (cols values of vec_dtype, each may be NULL) are overwritten,
 * or added to when accumulate is nonzero; with rows == 0 the sums are zero.
 * mean: NULL for MUON_NORM_RMS.  workspace: muon_norm_backward_workspace_bytes
 * bytes (needed only if dgamma or dbeta is given).  Errors as for
 * muon_norm_forward, and MUON_E_WORKSPACE. */
muon_status muon_norm_backward(int32_t kind, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               int64_t rows, int64_t cols, int32_t dtype, const void* gamma, int32_t vec_dtype,
                               const float* mean, const float* rstd, void* dx, int64_t lddx, void* dgamma,
                               void* dbeta, int32_t accumulate, void* workspace, size_t workspace_bytes,
                               void* stream);
muon_status muon_norm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes);

/* A linear layer y = x W^T + bias on 8-bit rows: x as tokens x in rows (q,
 * scale per token), W as out x in rows (wq, wscale per output channel).
 * The products of 8-bit values are summed exactly in 32-bit integers, hence
 * in <= 131071; with any scales that 8-bit rows have, a result in fp32's range
 * comes out finite.  y: tokens x out of dtype; bias: out values of bias_dtype,
 * or NULL.  The gradients are those of this layer with the rounding to 8 bits
 * taken as the identity:
 *   dW[n][k] = sum_t dy[t][n] scale[t] q[t][k]     out x in, dw_dtype; written,
 *              or added to dw when accumulate is nonzero
 *   dX[t][k] = sum_n dy[t][n] wscale[n] wq[n][k]   tokens x in, dx_dtype
 * dy: tokens x out, bf16 or fp32.  q * scale enters the gradient products in
 * bf16: exact for powers of two, rounded once for other scales.  fp32 dy is
 * taken as three bf16 pieces that add up to it: exactly from 2^-110 up, below
 * that without its bits under 2^-133, the last that bf16 has.
 * With tokens == 0 the weight gradient is zero; with out == 0 the input
 * gradient is; with in == 0 y is the bias (zero without one), whatever the
 * scales hold.
 * Errors: MUON_E_DTYPE; MUON_E_SHAPE (a size negative or above 2^30, in above
 * 131071 for the forward product, a leading dimension below its column count
 * or above 2^21, ldq or ldw not a multiple of 16, a result of more than 2^22
 * tiles, which are 128 x 128 or, of some large products, 256 x 256);
 * MUON_E_ARG (a pointer null or misaligned: 8-bit rows to 16 bytes, others to
 * their element);
 * MUON_E_WORKSPACE (workspace smaller than muon_linear8_workspace_bytes);
 * MUON_E_HIP. */
typedef enum {
  MUON_LINEAR8_FORWARD = 0,
  MUON_LINEAR8_WEIGHT_GRAD = 1,
  MUON_LINEAR8_INPUT_GRAD = 2
} muon_linear8_pass;
muon_status muon_linear8_forward(const int8_t* q, int64_t ldq, const float* scale, const int8_t* wq, int64_t ldw,
                                 const float* wscale, const void* bias, int32_t bias_dtype, int64_t tokens,
                                 int64_t out, int64_t in, void* y, int64_t ldy, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, void* stream);
muon_status muon_linear8_weight_grad(const void* dy, int64_t lddy, int32_t dy_dtype, const int8_t* q, int64_t ldq,
                                     const float* scale, int64_t tokens, int64_t out, int64_t in, void* dw,
                                     int64_t lddw, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                     size_t workspace_bytes, void* stream);
muon_status muon_linear8_input_grad(const void* dy, int64_t lddy, int32_t dy_dtype, const int8_t* wq, int64_t ldw,
                                    const float* wscale, int64_t tokens, int64_t out, int64_t in, void* dx,
                                    int64_t lddx, int32_t dx_dtype, void* workspace, size_t workspace_bytes,
                                    void* stream);
/* Bytes of workspace of one pass (muon_linear8_pass), host only; 0 for many
 * sizes, among them the forward pass of up to 16 tokens.  dy, lddy, dy_dtype:
 * those of the gradient call (the address is only looked at for its alignment:
 * bf16 dy whose rows are not whole 16-byte pieces, and fp32 dy where many
 * columns of the result share it, are laid out in the workspace first); ignored
 * for the forward pass.  Errors: MUON_E_METHOD (unknown pass), MUON_E_DTYPE,
 * MUON_E_SHAPE, MUON_E_ARG. */
muon_status muon_linear8_workspace_bytes(int32_t pass, int64_t tokens, int64_t out, int64_t in, const void* dy,
                                         int64_t lddy, int32_t dy_dtype, size_t* bytes);

/* Matrix products grouped by expert: rows offsets[e] .. offsets[e+1]-1 of x, y,
 * dy and dx belong to expert e, whose weight W[e] is out x in at
 * w + e * stride (elements), rows ldw apart:
 *   muon_experts_forward      y[r]  = x[r] W[e]^T                  rows x out
 *   muon_experts_input_grad   dx[r] = dy[r] W[e]                   rows x in
 *   muon_experts_weight_grad  dW[e] = sum over e's rows r of dy[r]^T x[r]
 * dW is laid out like W: with stride = out * lddw, lddw = in it is the gradient
 * of a Muon parameter of experts * out rows, split_rows = out, as muon_step
 * reads it.  dW is written, or added to when accumulate is nonzero; an expert
 * without rows gets zero (or what it had).
 * offsets: device memory, experts + 1 int32, 0 <= offsets[0] <= ... <=
 * offsets[experts] <= rows; read when the work runs, so a router on the device
 * may have written them just before on the same stream.  Rows before
 * offsets[0] and from offsets[experts] on belong to nobody: they are not read, and
 * y and dx are left as they were there.  Offsets outside 0 .. rows are taken as
 * the nearest of these; where they decrease, the results are unspecified, but
 * nothing outside the buffers is read or written.
 * dtype: of both operands; the results have their own.  bf16 products are
 * exact and summed in fp32; fp32 is multiplied and summed in fp32.
 * With in == 0 y is zero, with out == 0 dx is zero, with rows == 0 dW is zero
 * (or what it had).
 * The results overlap no operand, and calls that may run at the same time (two
 * streams, two graphs) have workspaces of their own.
 * Errors: MUON_E_DTYPE; MUON_E_SHAPE (a size negative, rows above 2^30, experts
 * above 2^16, a leading dimension below its column count or above 2^21, a
 * stride whose experts overlap or above 2^42, a result that may take more than
 * 2^22 tiles of 128 x 128); MUON_E_ARG (a pointer null or not aligned
 * to its element); MUON_E_WORKSPACE (smaller than
 * muon_experts_workspace_bytes); MUON_E_HIP. */
typedef enum {
  MUON_EXPERTS_FORWARD = 0,
  MUON_EXPERTS_WEIGHT_GRAD = 1,
  MUON_EXPERTS_INPUT_GRAD = 2
} muon_experts_pass;
muon_status muon_experts_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride,
                                 const int32_t* offsets, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                 int32_t dtype, void* y, int64_t ldy, int32_t y_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream);
muon_status muon_experts_input_grad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t stride,
                                    const int32_t* offsets, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                    int32_t dtype, void* dx, int64_t lddx, int32_t dx_dtype, void* workspace,
                                    size_t workspace_bytes, void* stream);
muon_status muon_experts_weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const int32_t* offsets,
                                     int64_t rows, int64_t experts, int64_t out, int64_t in, int32_t dtype, void* dw,
                                     int64_t lddw, int64_t stride, int32_t dw_dtype, int32_t accumulate,
                                     void* workspace, size_t workspace_bytes, void* stream);
/* Bytes of workspace of one pass (muon_experts_pass), host only, whatever the
 * operands' alignment: partial sums of products whose tiles are too few or too
 * unequal to fill the GPU, lists of the tiles of large ones, or 0.  Not an error
 * where out, in or rows is 0.  Errors: MUON_E_METHOD (unknown pass),
 * MUON_E_DTYPE, MUON_E_SHAPE, MUON_E_ARG. */
muon_status muon_experts_workspace_bytes(int32_t pass, int64_t rows, int64_t experts, int64_t out, int64_t in,
                                         int32_t dtype, size_t* bytes);

/* Static text for a status code. */
const char* muon_status_string(int32_t status);

/* Library version (major*10000 + minor*100 + patch). */
int32_t muon_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LIBMUON_H */
