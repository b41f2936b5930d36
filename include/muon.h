/*
 * libmuon -- the Muon optimizer step's hot path on AMD Instinct MI355X (gfx950).
 *
 * The step, per whole 2D weight matrix (blog "Muon Optimizer + FSDP",
 * section "Background: the conflict between FSDP and Muon"), in three calls:
 *   - refresh the momentum from the gradient   -> muon_momentum_update
 *                                                 (_sq: also the sums of
 *                                                 squares for the norms)
 *   - orthogonalise it by Newton-Schulz        -> muon_newton_schulz_batched
 *   - move the weight by -lr times the result  -> muon_apply
 * and, in front of it in a post-training step:
 *   - log-probabilities of tokens from logits  -> muon_token_logps
 *   - the loss with the gradient of the logits -> muon_policy_loss,
 *                                                 muon_preference_loss
 *   - the global gradient norm and clipping    -> muon_grad_norm,
 *                                                 muon_scale_grads,
 *                                                 muon_momentum_update_clipped
 *
 * Conventions shared by every entry point
 *   - Tensor arguments are DEVICE pointers to memory the caller owns and
 *     keeps alive until the work enqueued on `stream` has finished.  Matrices
 *     are dense row-major (rows x cols, leading dimension = cols).
 *   - `stream` is a hipStream_t passed as void* (NULL = the legacy default
 *     stream of the context's device).  Every call only enqueues work; none
 *     synchronises the device, none allocates device memory.
 *   - Arguments are validated before anything is enqueued: on any status
 *     other than MUON_OK nothing was launched.  Faults inside kernels surface
 *     at the caller's next synchronisation, as for any HIP kernel.
 *   - No C++ exception crosses this boundary.
 *   - A context is not thread-safe; use one context per stream (calls made
 *     on different streams with one context must be ordered by the caller).
 */
#ifndef LIBMUON_MUON_H
#define LIBMUON_MUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_EINVAL = 1,      /* null pointer, bad count/size, aliasing, bad parameter */
  MUON_ESHAPE = 2,      /* rows/cols <= 0, rows % head_rows != 0, ...           */
  MUON_EDTYPE = 3,      /* dtype or dtype combination not supported             */
  MUON_EWORKSPACE = 4,  /* the call needs more workspace than the context holds */
  MUON_EHIP = 5,        /* a HIP runtime call failed (see muon_last_error)      */
  MUON_ENOMEM = 6       /* host-side allocation failed                          */
} muon_status_t;

typedef enum { MUON_F32 = 0, MUON_BF16 = 1 } muon_dtype_t;

/* Elements per sum-of-squares partial (muon_momentum_update_sq). */
#define MUON_SQ_BLOCK 4096

/* How the iteration is evaluated (the DeepSpeed PR "[Muon] CPU offload: pin
 * the momentum and overlap the host writeback", section Tests, and the RFC's
 * section 5 Roadmap name an ns_method option with a "gram" choice beside the
 * standard one; neither page spells gram out).
 *   MUON_NS_QUINTIC: the iteration below on the m x n iterate, step by step.
 *   MUON_NS_GRAM:    the same polynomial map carried on m x m matrices only.
 *     With A_0 = X_0 X_0^T and P_k = a I + b A_k + c A_k^2 (a polynomial in
 *     A_k, so symmetric and commuting with it), X_{k+1} = P_k X_k gives
 *     A_{k+1} = P_k A_k P_k and X_steps = (P_{steps-1} ... P_0) X_0.  The
 *     m x n matrix is read twice (A_0 and the final product) instead of three
 *     times per step; every other product is m x m.  The result equals the
 *     quintic's in exact arithmetic; bf16 rounding differs.  A_0 carries the
 *     squared singular values, which bf16 resolves only when the matrix is
 *     far from square: in BF16 compute the Gram form runs on units with
 *     2 m <= n and the quintic iteration on the others (F32: always). */
typedef enum { MUON_NS_QUINTIC = 0, MUON_NS_GRAM = 1 } muon_ns_method_t;

/* Whole-iteration fusion for small units: a wide BF16 unit with m <= 128
 * (e.g. the 128 x n heads of per-head Muon, RFC section 4D) can run every
 * iteration in one launch, one workgroup per unit holding A and B (and, for
 * MUON_NS_GRAM, the m x m iterates) in on-chip memory.  The quintic
 * accumulates the next iteration's Gram product while the update is stored,
 * so the iterate is read once and written once per iteration; the Gram form
 * reads the input twice and writes the result once in all.  Results are
 * bit-identical to the unfused kernels.  AUTO fuses when the call has at
 * least as many units as the device has compute units (every CU gets a
 * unit), or when n <= 3072 (a workgroup then finishes its unit before the
 * separate launches would, however many CUs stay idle); ON whenever
 * eligible; OFF never.  Not eligible: tall units, m < 16 (those run in
 * fp32, see muon_newton_schulz_batched), m > 128, F32 compute, a
 * per-iteration coefficient table of more than
 * MUON_NS_FUSED_MAX_ROWS rows, and outputs that overlap an input other than
 * their own (in place, unit for unit, is fine). */
typedef enum { MUON_FUSE_AUTO = 0, MUON_FUSE_OFF = 1, MUON_FUSE_ON = 2 } muon_fuse_t;
#define MUON_NS_FUSED_MAX_ROWS 16

/* Newton-Schulz parameters.  The quintic iteration is the one the DeepSpeed
 * RFC "Enable Correct and High-Performance Muon Optimizer under ZeRO CPU
 * Offload" calls the current default (section 5, Roadmap), run for five to
 * six iterations (section 2, Root Cause Analysis).  Per iteration, on the
 * normalised matrix X (m x n, m <= n):
 *     A = X X^T ;  B = b A + c A A ;  X <- a X + B X
 * (the library forms B' = a I + B and computes X <- B' X, the same product
 * with one operand fewer).
 * X_0 = Y / (||Y||_F + eps); a tall Y (rows > cols) is processed as Y^T and
 * the result transposed back.  Defaults (muon_ns_params_default):
 * steps 5, (a, b, c) = (3.4445, -4.7750, 2.0315), eps 1e-7, compute BF16,
 * coeffs NULL.
 * Per-iteration coefficients (RFC section 5, Roadmap: coefficients optimised
 * for each iteration, "Polar Express"): when coeffs is not NULL it points to
 * `steps` rows of three floats (a_k, b_k, c_k), row-major, in HOST memory,
 * read during the call only; iteration k uses row k in place of (a, b, c)
 * (Gram form: P_k = a_k I + b_k A_k + c_k A_k^2).  Every value must be
 * finite.  muon_ns_minimax_coeffs fills such a table. */
typedef struct {
  int32_t steps;     /* >= 0 */
  float a, b, c;     /* quintic coefficients */
  float eps;         /* added to the Frobenius norm, >= 0 */
  int32_t compute;   /* muon_dtype_t: BF16 = bf16 MFMA with fp32 accumulate,
                        F32 = fp32 verification mode */
  int32_t method;    /* muon_ns_method_t, default MUON_NS_QUINTIC */
  int32_t fuse;      /* muon_fuse_t, default MUON_FUSE_AUTO */
  const float* coeffs; /* NULL, or steps x 3 per-iteration (a, b, c), host */
  /* Norms from the momentum pass (see muon_momentum_update_sq): NULL, or the
   * DEVICE array of sq_count partials that pass wrote for the update buffer
   * starting at the device address sq_base.  Every unit must then begin
   * sq_base + a whole number of MUON_SQ_BLOCK elements and span whole blocks
   * (its elements a multiple of MUON_SQ_BLOCK), inside the sq_count blocks;
   * its norm is the sum of its blocks' partials (fixed order) and the inputs
   * are not read for it.  The partials must describe the current contents of
   * the units (the caller's ordering).  Violations: MUON_EINVAL. */
  const double* sq_partials;
  const void* sq_base;
  int64_t sq_count;
} muon_ns_params_t;

/* Geometry of one weight matrix (RFC section 4A: keep the 2D shape and head
 * dimensions with the parameter).  head_rows = 0: the whole matrix is one
 * Newton-Schulz unit; head_rows = h > 0: rows/h contiguous row blocks of
 * h x cols are orthogonalised independently (RFC section 4D, per-head Muon;
 * blog section "Chunked communication": split fused tensors into their
 * logical matrices, never row-split one matrix). */
typedef struct {
  int64_t rows, cols, head_rows;
} muon_shape_t;

typedef struct muon_ctx muon_ctx_t;
typedef struct muon_plan_s muon_plan_t;

/* ------------------------------------------------------------------------ */
/* Context and workspace                                                     */
/* ------------------------------------------------------------------------ */

/* Create a context on HIP device `device` holding one preallocated device
 * workspace slab of `workspace_bytes` (blog section "Memory control", item 2:
 * preallocate the workspace once and only take views of it per micro-bucket),
 * and beside it 265 KiB through which the workgroups of one loss call exchange
 * what they found.  This is the only call that allocates device memory.  It
 * waits for the device's null stream, so that the context is ready for every
 * stream.  On success *out owns the slab until muon_destroy.  Errors: MUON_EINVAL (out NULL),
 * MUON_EHIP (no such device / allocation failed), MUON_ENOMEM. */
muon_status_t muon_create(int device, size_t workspace_bytes, muon_ctx_t** out);

/* Free the context and its workspace (blog section "Memory control", item 2:
 * the workspace lives as long as the context).  Waits for the context's
 * device to finish the work enqueued so far.  NULL is accepted. */
muon_status_t muon_destroy(muon_ctx_t* ctx);

/* Size of the context's workspace slab in bytes (0 for NULL; blog section
 * "Memory control", item 2). */
size_t muon_ctx_workspace_bytes(const muon_ctx_t* ctx);

/* Fill *p with the defaults listed above (RFC section 5, Roadmap: the
 * quintic iteration is the current default; section 2: five to six
 * iterations). */
void muon_ns_params_default(muon_ns_params_t* p);

/* Per-iteration coefficients (RFC section 5, Roadmap: Newton-Schulz with
 * coefficients optimised per iteration, so that fewer iterations reach the
 * same accuracy; the page gives no table).  Iteration t maps each singular
 * value x to p_t(x) = a x + b x^3 + c x^5, where p_t is the odd quintic with
 * the smallest max |1 - p(x)| over [l_t, u_t (1 + margin)], the interval
 * that holds the singular values at that point; l_0 = lo, u_0 = 1 (X_0 is
 * normalised by its Frobenius norm), and the next interval is p_t's image
 * [1 - E_t, 1 + E_t], E_t the attained maximum.  `margin` widens each
 * interval at the top, where p_t climbs steeply, so that values that bf16
 * rounding pushes slightly past it stay bounded and rounding errors near
 * the top are amplified less (0.05 is the binding's default: a few bf16
 * roundings of 2^-8 each, with room).  An interval narrower than 1e-3 takes the limit
 * polynomial (15/8, -5/4, 3/8).  Pure host function, computed in double.
 * out: `steps` x 3 floats (caller-owned, host).  *bound (may be NULL)
 * receives E_{steps-1}: in exact arithmetic every singular value of X_0 in
 * [lo, 1] ends within [1 - bound, 1 + bound].  `margin` must lie in [0.01, 0.1]:
 * with bf16 iterates, low-rank inputs reached relative errors of 0.36 at
 * margin 0 and 0.14 at margin 0.2 against the fp64 iteration with the same
 * coefficients, and stayed within 2e-2 inside that window.  Errors:
 * MUON_EINVAL (steps < 1 or > 1024, lo outside (0, 1), margin outside
 * [0.01, 0.1], out NULL, or the exchange did not converge). */
muon_status_t muon_ns_minimax_coeffs(int32_t steps, double lo, double margin, float* out,
                                     double* bound);

/* Workspace one muon_newton_schulz_batched call needs for `count` matrices
 * of `shape` in compute dtype `compute` (pure host function; blog section
 * "Memory control", item 2).  Per Newton-Schulz unit of m x n (m = min, n =
 * max of its rows and cols, e = element bytes of the compute dtype): two
 * iterate buffers (2 e m n) + A and B (2 e m^2) + 8 bytes of scalars + 8
 * bytes per norm partial (at most 512); in BF16 also the iterate's rounding
 * residual (2 bytes per element, rows and columns padded to the tile: 256
 * once m >= 256, else 128) and B's diagonal in fp32 (4 m).  Each region is
 * rounded up to 256 bytes: (2 + 2 m/n) x the unit's e m n bytes (BF16:
 * 3 + 2 m/n, up to the residual's padding) plus scalars.  BF16 units with
 * m < 16 run the iteration in fp32: for them it is at least the inputs
 * widened to fp32 (4 m n) plus the F32 figure.  Returns 0 for an invalid
 * shape or count <= 0. */
size_t muon_ns_workspace_bytes(muon_shape_t shape, int64_t count, int32_t compute);

/* Workspace to run Newton-Schulz over a list of matrices of mixed shapes,
 * one muon_newton_schulz_batched call per group of identical shapes
 * (rows, cols, head_rows), the calls one after another on one context: the
 * largest group's muon_ns_workspace_bytes (blog section "Memory control",
 * item 2: the workspace is a stated function of what one call holds).  Pure
 * host function.  Returns 0 when count <= 0 or a shape is invalid. */
size_t muon_workspace_bytes(const muon_shape_t* shapes, int64_t count, int32_t compute);

/* ------------------------------------------------------------------------ */
/* Host scheduler: same-shape buckets split into micro-buckets under a cap   */
/* ------------------------------------------------------------------------ */

typedef enum {
  MUON_CAP_FULL_BYTES = 0,  /* sum of full-matrix bytes (e * rows * cols) <= cap */
  MUON_CAP_WORKSPACE = 1    /* sum of Newton-Schulz workspace bytes      <= cap */
} muon_cap_kind_t;

typedef struct {
  int64_t m, n;               /* canonical shape of the bucket's units (m <= n) */
  int64_t count;              /* matrices in this micro-bucket                 */
  int64_t units;              /* Newton-Schulz units (heads expanded)          */
  int64_t numel;              /* elements of its matrices                      */
  size_t full_bytes;          /* e * numel                                      */
  size_t workspace_bytes;     /* sum of muon_ns_workspace_bytes per shape group */
  int32_t over_cap;           /* 1 if a single matrix alone exceeds the cap     */
  int32_t shape_groups;       /* distinct (rows, cols, head_rows) runs inside   */
  int64_t elem_offset;        /* its first element in the plan's flat layout   */
} muon_bucket_info_t;

/* Group `count` matrices into buckets by canonical unit shape (m, n) in order
 * of first appearance (blog section "Memory control", item 6: merge same-shape
 * matrices across layers into one bucket), order each bucket's members by
 * orientation (units of the first member's orientation first: wide units,
 * rows <= cols, and tall ones run separate launches) and then by exact shape
 * (stable), so that members whose units share a shape lie together, and cut
 * each bucket into micro-buckets of whole
 * matrices whose cost stays within `cap_bytes` (blog sections "Chunked
 * communication" and "Memory control", item 1: a separate Muon cap;
 * estimate_muon_peak(bucket) <= cap).  A matrix larger than the cap gets a
 * micro-bucket of its own, flagged over_cap.
 * compute_units = 0: micro-buckets are filled greedily up to the cap.
 * compute_units = C > 0 (the device's CU count): the cut points are chosen,
 * still under the cap, to minimise a model of the Newton-Schulz time on C
 * CUs -- each product launch takes ceil(tiles / slots) rounds of its
 * per-tile k-length (one 256-tile per CU, or two 128-tiles per CU at 0.6 of
 * a 256-tile round where the launch takes those because few 256-tiles would
 * leave most CUs idle), each orientation of a micro-bucket its own
 * launches -- plus a
 * fixed cost per launch chain, so that launches do not end with a nearly
 * empty last round of tiles.  Host only; *out is owned by the
 * caller (muon_plan_destroy).  Errors: MUON_EINVAL, MUON_ESHAPE. */
muon_status_t muon_plan_create(const muon_shape_t* shapes, int64_t count, size_t cap_bytes,
                               int32_t cap_kind, int32_t compute, int32_t compute_units,
                               muon_plan_t** out);
/* muon_plan_create with BF16 compute and the plain cap-filling cuts
 * (compute_units = 0): the scheduler's signature with the cap and its kind
 * only (blog sections "Chunked communication" and "Memory control", items 1
 * and 6). */
muon_status_t muon_plan(const muon_shape_t* shapes, int64_t count, size_t cap_bytes,
                        int32_t cap_kind, muon_plan_t** out);
/* Number of micro-buckets (blog section "Chunked communication"). */
int64_t muon_plan_num_buckets(const muon_plan_t* plan);
/* Info on micro-bucket `b`.  When non-NULL, `indices` receives info->count
 * matrix indices (positions in the `shapes` array) in execution order, and
 * `offsets` the element offset of each of those matrices in the plan's flat
 * layout: state buffers (gradients, momentum, weights) that hold every matrix
 * in plan order -- micro-bucket after micro-bucket, members packed in
 * execution order -- so that each micro-bucket is one contiguous range
 * starting at info->elem_offset (blog section "DBuffer": addresses planned
 * once at init, views per step).  Errors: MUON_EINVAL (NULL plan or info, b
 * out of range). */
muon_status_t muon_plan_bucket(const muon_plan_t* plan, int64_t b, muon_bucket_info_t* info,
                               int64_t* indices, int64_t* offsets);
/* Elements of the plan's flat layout (the sum of every matrix's rows x cols;
 * blog section "DBuffer": one persistent buffer per state). */
int64_t muon_plan_total_elems(const muon_plan_t* plan);
/* Largest workspace_bytes over the plan's micro-buckets: a context this large
 * runs every micro-bucket (blog section "Memory control", item 2: one
 * preallocated workspace sized by the cap). */
size_t muon_plan_max_workspace(const muon_plan_t* plan);
/* Free a plan (NULL is accepted; blog section "Memory control": the plan is
 * made once at init and kept). */
void muon_plan_destroy(muon_plan_t* plan);

/* ------------------------------------------------------------------------ */
/* The three steps                                                           */
/* ------------------------------------------------------------------------ */

/* Momentum with Nesterov look-ahead over `numel` contiguous elements
 * (blog, section "Background": the momentum refresh; RFC section 2:
 * the first-order momentum the offload path must keep).  Per element, each
 * operation one IEEE binary32 rounding, no fused multiply-add:
 *     t  = (1 - beta) * g
 *     M' = beta * M + t                      (written back to momentum)
 *     U  = t + beta * M'   (nesterov != 0)   or   U = M'   (nesterov == 0)
 * grad: `grad_dtype` (BF16 or F32); momentum: F32, updated in place;
 * update_out: `update_dtype` (BF16 = U rounded to nearest-even, or F32).
 * numel == 0 is a no-op.  update_out may not alias grad or momentum; all
 * pointers must be element-aligned.  Errors: MUON_EINVAL (NULL pointer,
 * numel < 0, aliasing, beta outside [0, 1]), MUON_EDTYPE, MUON_EHIP. */
muon_status_t muon_momentum_update(muon_ctx_t* ctx, void* stream, const void* grad,
                                   int32_t grad_dtype, float* momentum, void* update_out,
                                   int32_t update_dtype, int64_t numel, float beta,
                                   int32_t nesterov);

/* muon_momentum_update, which also leaves the sums of squares that the
 * Newton-Schulz normalisation X_0 = U / (||U||_F + eps) needs (blog section
 * "Background": Newton-Schulz runs on the refreshed momentum; the sums of
 * squares come out of the same pass, so the Frobenius norms need no second
 * read of U).  sq_partials (device,
 * ceil(numel / MUON_SQ_BLOCK) doubles, caller-owned) receives for block b the
 * sum of squares of update elements [b*4096, min((b+1)*4096, numel)) as
 * stored (bf16 values when update_dtype is BF16), in binary64: every square
 * is exact, the sum runs in a fixed order, so the partials are reproducible
 * bit for bit.  Pass them to muon_newton_schulz_batched through
 * muon_ns_params_t.sq_partials.  Errors: those of muon_momentum_update, and
 * MUON_EINVAL for a NULL or overlapping sq_partials. */
muon_status_t muon_momentum_update_sq(muon_ctx_t* ctx, void* stream, const void* grad,
                                      int32_t grad_dtype, float* momentum, void* update_out,
                                      int32_t update_dtype, int64_t numel, float beta,
                                      int32_t nesterov, double* sq_partials);

/* Batched Newton-Schulz over one same-shape group (blog section "Chunked
 * communication": every Muon unit stays a whole matrix; XTuner-style same-
 * shape buckets).  mats: HOST array of `count` device pointers to rows x cols
 * matrices of io_dtype; out: HOST array of `count` device pointers receiving
 * the orthogonalised update in the same shape and dtype (out == NULL, or
 * out[i] == mats[i], means in place).  With shape.head_rows = h > 0 every
 * h x cols row block is orthogonalised on its own.  Supported (io_dtype,
 * params->compute): (BF16, BF16) -- bf16 MFMA, fp32 accumulate, A, B and
 * the X iterates rounded to bf16 (units whose smaller side is under 16:
 * the iteration in fp32 on widened inputs, the result rounded to bf16);
 * (F32, F32) -- fp32 verification mode.
 * The Frobenius norm is reduced deterministically (fixed order), so two
 * calls on identical inputs give identical bits.  A unit whose norm is 0
 * yields exactly 0.  nonfinite_flag (device int, may be NULL) gets 1 OR-ed
 * in when some unit's norm is not finite; values are propagated, never
 * skipped.  Uses the context workspace (muon_ns_workspace_bytes(shape,
 * count, compute) bytes).  count == 0 is a no-op.  The call may be recorded
 * into a HIP graph (stream capture) when the inputs, and the outputs, are
 * evenly spaced; irregularly placed matrices need pointer tables uploaded
 * from a host ring that later calls reuse, and are rejected while the
 * stream captures (MUON_EINVAL).  Errors: MUON_EINVAL, MUON_ESHAPE,
 * MUON_EDTYPE, MUON_EWORKSPACE, MUON_EHIP. */
muon_status_t muon_newton_schulz_batched(muon_ctx_t* ctx, void* stream, const void* const* mats,
                                         int64_t count, muon_shape_t shape, int32_t io_dtype,
                                         const muon_ns_params_t* params, void* const* out,
                                         int* nonfinite_flag);

/* Weight apply over `numel` contiguous elements (blog, section "Background":
 * the weight moves by -lr times the orthogonalised update).  Each
 * operation one binary32 rounding, no FMA:
 *     eta = lr * scale;  W1 = W * (1 - lr * weight_decay) if weight_decay != 0
 *     W'  = W1 - eta * u                        (written back to master)
 *     weight_bf16 = W' rounded to nearest-even  (when weight_bf16 != NULL)
 * update: `update_dtype` (BF16 or F32).  numel == 0 is a no-op.
 * Errors: MUON_EINVAL (NULL master/update, numel < 0, aliasing),
 * MUON_EDTYPE, MUON_EHIP. */
muon_status_t muon_apply(muon_ctx_t* ctx, void* stream, float* master, const void* update,
                         int32_t update_dtype, void* weight_bf16, int64_t numel, float lr,
                         float scale, float weight_decay);

/* Allocation-free Newton-Schulz, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments, kernels and results as
 * muon_newton_schulz_batched (bit for bit), without a context: the workspace
 * is a static device array of MUON_NOALLOC_SCRATCH_BYTES that every GPU the
 * library runs on holds from the first call there until the process ends
 * (the first call on a device looks its address up; no call allocates).
 * device: the HIP device the stream belongs to.  The call's workspace
 * (muon_ns_workspace_bytes(shape, count, params->compute)) must fit the
 * scratch, else MUON_EWORKSPACE.  Matrices must be evenly spaced (mats[i] =
 * mats[0] + i * d, no overlap), and out NULL (in place), equal to mats, or
 * evenly spaced and disjoint from every input; otherwise MUON_EINVAL.  Every
 * call on one GPU shares that GPU's scratch: calls that overlap on one GPU
 * (different streams or threads, without ordering) race and give undefined
 * results.  No per-kernel timing.  muon_noalloc_last_error() gives the
 * calling thread's last error text (a static string). */
#define MUON_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
muon_status_t muon_newton_schulz_batched_noalloc(int device, void* stream,
                                                 const void* const* mats, int64_t count,
                                                 muon_shape_t shape, int32_t io_dtype,
                                                 const muon_ns_params_t* params,
                                                 void* const* out, int* nonfinite_flag);
const char* muon_noalloc_last_error(void);

/* ------------------------------------------------------------------------ */
/* The losses in front of the step: log-probabilities of chosen tokens       */
/* ------------------------------------------------------------------------ */

/* A batch of rows of scores over a vocabulary: element (b, t, v) at data +
 * (b * batch_stride + t * row_stride + v) elements of `dtype`; strides in
 * elements, so that a padded vocabulary (row_stride > vocab), logits shifted
 * against their labels (a batch_stride longer than seq rows) and sequence-major
 * storage are all described without a copy.  Inputs may overlap themselves
 * (strides of 0 included); rows that are written must be disjoint.  Strides
 * are >= 0; that of a dimension of size one is ignored. */
#define MUON_MAX_VOCAB (1 << 19)
typedef struct {
  void* data;
  int32_t dtype;                    /* MUON_BF16 or MUON_F32 */
  int64_t batch, seq, vocab;        /* vocab in [1, MUON_MAX_VOCAB], batch * seq <= 2^30 */
  int64_t batch_stride, row_stride; /* elements */
} muon_logits_t;

/* Conventions of the calls below, beside those of every entry point.
 *   - R = batch * seq tokens; arrays "per token" are dense [batch][seq].
 *   - labels (device, int64 per token): the chosen token of each row.  A
 *     negative label leaves the token out: its row is not read, nothing of it
 *     enters a sum (whatever the other per-token inputs hold there), its
 *     log-probability is 0 and its gradient row is zeros.  A label >= vocab
 *     names no score: the token's log-probability and gradient are NaN.
 *   - z = x / temperature are the scores that the softmax sees; temperature
 *     in (1e-30, 1e30).  Scores of -infinity have probability 0; a row of
 *     nothing else, or with NaN or +infinity in it, gives NaN, as the formula
 *     does.
 *   - Sums over a vocabulary run in a fixed order around the row's maximum:
 *     fp32 exponentials, added in fp32 by fours (fp32 scores) or eights (bf16)
 *     and in binary64 beyond, so that small log-probabilities keep their
 *     relative accuracy too.  Log-probabilities are formed, and everything per
 *     token or sequence summed, in binary64 and rounded to fp32 when stored.
 *     Two calls on identical inputs, rows at the same alignment to 16 bytes,
 *     give identical bits.
 *   - Gradients are of `weight` times the loss with respect to x and have
 *     x's dtype (fp32 arithmetic, one rounding).  They may replace the scores
 *     in place (same address, strides and dtype); any other overlap between
 *     what a call writes and what it reads or also writes is refused.
 *   - The context's workspace holds what the kernels hand each other
 *     (muon_loss_workspace_bytes), so calls on one context are ordered.  Every
 *     call may be recorded into a HIP graph.
 * Errors of all of them: MUON_EINVAL (ctx or another required pointer NULL,
 * misaligned pointers, bad parameters, overlaps), MUON_ESHAPE, MUON_EDTYPE,
 * MUON_EWORKSPACE, MUON_EHIP.  A batch or seq of 0 is no error: the losses of
 * no token follow (and 0 for no pair), per-token arrays are empty and may be
 * NULL. */

/* Workspace in bytes of any one of the loss calls on batch x seq rows of
 * `vocab` scores of `dtype` (pure host function; 0 for arguments out of
 * range).  8 bytes per row and slice of a row, 32 per row beside. */
size_t muon_loss_workspace_bytes(int64_t batch, int64_t seq, int64_t vocab, int32_t dtype);

/* Log-probability of every token: logps[t] = z[y] - log sum_v exp(z[v]).
 * logps: fp32 per token.  row_stats (may be NULL): two floats per token, the
 * row's maximum score and its sum of exponentials around it less 1, which
 * muon_token_logps_backward takes. */
muon_status_t muon_token_logps(muon_ctx_t* ctx, void* stream, const muon_logits_t* logits,
                               const int64_t* labels, double temperature, float* logps,
                               float* row_stats);

/* Its gradient: grad_logits[t][v] = grad_logps[t] / temperature *
 * ([v = y] - exp(z[v]) / sum).  logits, labels, temperature as given to
 * muon_token_logps, row_stats as it left them. */
muon_status_t muon_token_logps_backward(muon_ctx_t* ctx, void* stream, const muon_logits_t* logits,
                                        const int64_t* labels, double temperature,
                                        const float* row_stats, const float* grad_logps,
                                        const muon_logits_t* grad_logits);

/* How the per-token terms l_t of the policy loss become one number.
 *   MUON_REDUCE_TOKEN:    sum_t l_t / N over the N tokens that count
 *   MUON_REDUCE_SEQUENCE: (1 / batch) sum_b (mean of l_t over b's tokens); a
 *                         sequence with no token contributes 0
 *   MUON_REDUCE_SUM:      sum_t l_t */
typedef enum {
  MUON_REDUCE_TOKEN = 0,
  MUON_REDUCE_SEQUENCE = 1,
  MUON_REDUCE_SUM = 2
} muon_reduce_t;

typedef struct {
  double temperature;
  float clip_low, clip_high;     /* ratio range [1 - clip_low, 1 + clip_high]; in [0, 1], >= 0 */
  float kl_coef;                 /* >= 0; > 0 needs ref_logps */
  float weight;                  /* factor of loss and gradient, e.g. 1 / accumulation steps */
  int32_t reduce;                /* muon_reduce_t */
  int32_t advantage_per_token;   /* advantages: 0 = [batch], 1 = per token */
} muon_policy_params_t;

/* Clipped policy loss with a KL term, and its gradient.  Per token that
 * counts, with lp the policy's log-probability, A its advantage:
 *     r  = exp(lp - old_logps)           (old_logps NULL: r = 1, its
 *                                         gradient that of lp - constant)
 *     pg = max(-A r, -A min(max(r, 1 - clip_low), 1 + clip_high))
 *     kl = exp(e) - 1 - e,  e = ref_logps - lp       (ref_logps NULL: 0)
 *     l  = pg + kl_coef kl,   dl/dlp = -A r [-A r >= the clipped one]
 *                                      + kl_coef (1 - exp(e))
 * out: four floats {weight * loss, and reduced as the loss is, without
 * `weight`: pg, kl, [the clipped term is the larger]}.  logps (may be NULL): the log-probabilities, fp32 per token.
 * grad_logits (may be NULL: no gradient is formed). */
muon_status_t muon_policy_loss(muon_ctx_t* ctx, void* stream, const muon_logits_t* logits,
                               const int64_t* labels, const muon_policy_params_t* params,
                               const float* advantages, const float* old_logps,
                               const float* ref_logps, float* out, float* logps,
                               const muon_logits_t* grad_logits);

/* MUON_PREFERENCE_SIGMOID: -(1 - s) log sigma(h) - s log sigma(-h), h = beta m
 *                          (s = 0: the first term alone, also where h is infinite)
 * MUON_PREFERENCE_IPO:     (m - 1 / (2 beta))^2 */
typedef enum { MUON_PREFERENCE_SIGMOID = 0, MUON_PREFERENCE_IPO = 1 } muon_preference_t;

typedef struct {
  double temperature;
  float beta;             /* > 0 */
  float label_smoothing;  /* s, in [0, 0.5]; sigmoid only (else 0) */
  float weight;           /* factor of loss and gradient */
  int32_t kind;           /* muon_preference_t */
  int32_t average;        /* 0: a sequence's score is the sum over its tokens, 1: the mean */
} muon_preference_params_t;

/* Preference loss over pairs, and its gradient.  batch = 2 P sequences:
 * sequence i < P was preferred over sequence P + i.  With s_i the sum (or the
 * mean) of lp - ref_logps over sequence i's tokens (ref_logps NULL: of lp; no
 * token: 0) and the margin m = s_i - s_{P+i}, the loss is the mean of the
 * pairs' terms (muon_preference_t).  out: three floats {weight * loss, mean of
 * beta m, share of pairs with m > 0}.  rewards (may be NULL): beta s_i, fp32
 * per sequence.  logps, grad_logits: as for muon_policy_loss.  An odd batch:
 * MUON_ESHAPE. */
muon_status_t muon_preference_loss(muon_ctx_t* ctx, void* stream, const muon_logits_t* logits,
                                   const int64_t* labels, const muon_preference_params_t* params,
                                   const float* ref_logps, float* out, float* rewards,
                                   float* logps, const muon_logits_t* grad_logits);

/* ------------------------------------------------------------------------ */
/* Global gradient norm and clipping                                         */
/* ------------------------------------------------------------------------ */

/* One tensor of a list: numel contiguous elements at data (device), aligned to
 * the element. */
typedef struct {
  void* data;
  int64_t numel;   /* in [0, 1.37e11] (2^37 - 2^14); 2^40 in a whole list */
  int32_t dtype;   /* MUON_BF16 or MUON_F32 */
} muon_tensor_t;

/* Workspace in bytes of muon_grad_norm over these tensors (host array; pure
 * host function; 0 when count <= 0 or an entry is invalid). */
size_t muon_grad_norm_workspace_bytes(const muon_tensor_t* grads, int64_t count);

/* Norm over all elements of `count` tensors of any mix of sizes and dtypes:
 * norm (device, three doubles) receives {S, sqrt(S), coefficient}, S the sum
 * of the squares of every element -- each square exact in binary64, summed in
 * a fixed order, so the result is reproducible bit for bit and nothing
 * overflows -- and coefficient = min(1, max_norm / (sqrt(S) + eps)), NaN when
 * S is NaN.  max_norm > 0 (infinity: the coefficient of a finite S is 1), eps
 * >= 0.  Where gradients are sharded, sum norm[0] over the ranks and call
 * muon_clip_coef.  The tensor list is read during the call only (host array);
 * it travels in kernel arguments, so the call may be recorded into a HIP
 * graph.  count == 0: S = 0.  Errors: MUON_EINVAL, MUON_ESHAPE (numel < 0 or
 * too large), MUON_EDTYPE, MUON_EWORKSPACE, MUON_EHIP. */
muon_status_t muon_grad_norm(muon_ctx_t* ctx, void* stream, const muon_tensor_t* grads,
                             int64_t count, double max_norm, double eps, double* norm);

/* norm[1] and norm[2] from norm[0] (device), as muon_grad_norm forms them. */
muon_status_t muon_clip_coef(muon_ctx_t* ctx, void* stream, double max_norm, double eps,
                             double* norm);

/* out[i] = c * grads[i] with c = norm[2] rounded to fp32 (device, read by the
 * kernels: no host synchronisation), each product rounded to fp32 and then to
 * out[i]'s dtype.  out NULL: in place; a coefficient of exactly 1 then writes
 * nothing.  Otherwise out[i] has grads[i]'s numel, any dtype, and is disjoint
 * from every other tensor of both lists (out[i] == grads[i], same dtype, is
 * in place); gradients that are only read may overlap each other.  Errors: as
 * for muon_grad_norm. */
muon_status_t muon_scale_grads(muon_ctx_t* ctx, void* stream, const muon_tensor_t* grads,
                               const muon_tensor_t* out, int64_t count, const double* norm);

/* muon_momentum_update_sq on the clipped gradient g' = c * g (one binary32
 * rounding), c = norm[2] rounded to binary32, norm as muon_grad_norm leaves it
 * on the device: the momentum pass reads the gradient anyway, so clipping
 * costs no pass of its own and the gradient stays as it is.  sq_partials may
 * be NULL (no partials).  Errors: those of muon_momentum_update_sq, and
 * MUON_EINVAL for a NULL or misaligned norm. */
muon_status_t muon_momentum_update_clipped(muon_ctx_t* ctx, void* stream, const void* grad,
                                           int32_t grad_dtype, float* momentum, void* update_out,
                                           int32_t update_dtype, int64_t numel, float beta,
                                           int32_t nesterov, const double* norm,
                                           double* sq_partials);

/* ------------------------------------------------------------------------ */
/* Diagnostics                                                               */
/* ------------------------------------------------------------------------ */

/* Static text for a status code ("unknown status" for values outside the
 * enum).  Error reporting is part of the per-bucket diagnostics the blog's
 * section "Metrics to record" asks for. */
const char* muon_status_string(muon_status_t s);
/* Text of the last error recorded on ctx (empty string when none), blog
 * section "Metrics to record".  NULL ctx: a static text, that of the calling
 * thread's last refusal of a call made without a context (empty when none). */
const char* muon_last_error(const muon_ctx_t* ctx);

/* Per-kernel-class timing with HIP events recorded on the launch stream
 * around each kernel (per-bucket timing, blog section "Metrics to record").
 * enable != 0 preallocates an event pool; launches beyond its capacity, and
 * launches recorded into a graph (stream capture), are not timed.  muon_timing_read synchronises on the recorded events and
 * returns the summed duration and number of timed launches of one class. */
typedef enum {
  MUON_K_MOMENTUM = 0,
  MUON_K_NORM = 1,
  MUON_K_GRAM = 2,
  MUON_K_SYMSQ = 3,
  MUON_K_UPDATE = 4,
  MUON_K_APPLY = 5,
  MUON_K_PROD = 6,   /* m x m products of MUON_NS_GRAM (P_k Q_k, P_k A_k, (P_k A_k) P_k) */
  MUON_K_FUSED = 7,  /* whole-iteration launches of small units (muon_fuse_t) */
  MUON_K_LOSS = 8,   /* token log-probabilities, the losses and their gradients */
  MUON_K_CLIP = 9,   /* global gradient norm and gradient scaling */
  MUON_K_COUNT = 10
} muon_kernel_class_t;

muon_status_t muon_timing_enable(muon_ctx_t* ctx, int32_t enable, int32_t capacity);
/* How often a workgroup of muon_policy_loss polls for what the other
 * workgroups of its row publish before it computes that itself (default
 * 16384, tens of milliseconds; the results are the same bits either way).
 * 0: at once.  Errors: MUON_EINVAL (ctx NULL, polls < 0). */
muon_status_t muon_loss_set_polls(muon_ctx_t* ctx, int32_t polls);
/* Time only the kernel classes whose bit (1u << muon_kernel_class_t) is set
 * in class_mask: launches of the other classes record no events, and so
 * add no event markers to their stream (every class is timed by default;
 * 0 times none).  Takes effect for launches enqueued after the call.
 * Errors: MUON_EINVAL (ctx NULL, or a bit at or above MUON_K_COUNT set). */
muon_status_t muon_timing_select(muon_ctx_t* ctx, uint32_t class_mask);
muon_status_t muon_timing_reset(muon_ctx_t* ctx);
muon_status_t muon_timing_read(muon_ctx_t* ctx, int32_t kernel_class, double* total_ms,
                               int64_t* launches);

#ifdef __cplusplus
}
#endif
#endif /* LIBMUON_MUON_H */
