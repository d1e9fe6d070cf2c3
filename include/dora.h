/*
 * libdora: the DoRA forward hot path on AMD Instinct MI355X (gfx950).
 *
 * DoRA writes an adapted weight as W' = m * (W + sBA) / ||W + sBA||_row
 * ("Scaling DoRA: High-Rank Adaptation via Factored Norms and Fused Kernels",
 * summary on alanhou.org, "The Problem"). This library computes the two
 * pieces of that forward pass that dominate its cost:
 *
 *   dora_factored_norm  the row norm ||W + sBA||_row without forming BA,
 *                       through ||W||^2 + 2s<W,BA> + s^2||BA||^2 with
 *                       U = W A^T and G = A A^T ("DoRA优化技术解析：从内存瓶颈到
 *                       高效实现", cyqw.cn, §1.2, §1.2.1, §5.1 Algorithm 1),
 *                       and optionally g = m / max(wnorm, eps) (same page,
 *                       §1.2.2);
 *   dora_compose        the stable magnitude compose
 *                       (g - 1) * base + g * (s * lora) in one pass
 *                       (same page, §2.1, §2.1.1, §5.2);
 *   dora_compose_backward
 *                       its gradients d_base, d_lora and dg (dm) in one
 *                       pass plus a deterministic column reduction (same
 *                       page, §4.2, §5.2, §6.1 Table 9).
 *
 * Conventions shared by every entry point:
 *   - Matrices are dense, row-major and contiguous. Layouts follow LoRA:
 *     W [d_out, d_in], A [r, d_in], B [d_out, r]; activations [T, d_out].
 *   - Device pointers are device memory the caller owns (e.g. torch
 *     tensors). The library allocates nothing and never frees or retains
 *     a pointer. Its only host state is the device address of the
 *     dora_factored_norm_noalloc scratch array on each GPU, looked up once
 *     per GPU and never changed.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream of
 *     the current GPU). The current GPU is the one that the stream and the
 *     buffers belong to.
 *     All work is enqueued asynchronously on it; results are valid once
 *     the stream has reached that point. Calls enqueue kernels only (no
 *     memset, copy, allocation or host synchronisation; counters a call
 *     needs are cleared by one of its own kernels), so a sequence of calls
 *     can be captured into a HIP graph and replayed; a replay depends on
 *     nothing an earlier call left in the workspace.
 *   - Errors: arguments are checked on the host before any launch. A
 *     failed check returns a non-zero dora_status and enqueues nothing.
 *     A HIP launch error returns DORA_ERR_HIP. No exception crosses this
 *     ABI and no call aborts the process.
 *   - Results are bitwise reproducible from run to run for the same
 *     arguments: reductions use a fixed order and no floating-point
 *     atomics.
 */
#ifndef DORA_H_
#define DORA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dora_status {
  DORA_OK = 0,
  DORA_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad alias  */
  DORA_ERR_UNSUPPORTED_DTYPE = 2, /* dtype code not in dora_dtype            */
  DORA_ERR_BUDGET = 3,            /* workspace needed exceeds the budget     */
  DORA_ERR_WORKSPACE = 4,         /* workspace pointer too small / misaligned */
  DORA_ERR_HIP = 5                /* a HIP runtime or launch call failed     */
} dora_status;

typedef enum dora_dtype {
  DORA_BF16 = 0, /* bfloat16 storage, fp32 arithmetic */
  DORA_F32 = 1,  /* binary32 storage and arithmetic   */
  DORA_F16 = 2   /* binary16 storage, fp32 arithmetic (accumulation in fp32;
                    G = A A^T, which may exceed binary16's range, is held as
                    bf16 hi + lo or in fp32) */
} dora_dtype;

/* 8-bit operands of dora_matmul and the 8-bit output of dora_rms_norm: OCP
 * e4m3 (largest value 448, no infinity). No other entry point takes it. */
#define DORA_E4M3 3

/* Human-readable name of a status code (static string, never NULL). */
const char* dora_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int dora_version(void);

/*
 * Chunk width of the factored norm's d_in loop, as the cyqw.cn page defines
 * it (§5.1 Algorithm 1, step 1): the fp32 chunk buffer [d_out, cs] must fit
 * `budget_bytes`, aligned to 64 elements. cs = min(d_in, max(64,
 * 64 * floor(floor(budget / (4 d_out)) / 64))); cs = d_in when d_out or
 * d_in is 0. Host only; never touches the GPU.
 * Returns DORA_ERR_INVALID_ARG for negative sizes or cs == NULL.
 */
dora_status dora_norm_chunk_size(int64_t d_out, int64_t d_in, size_t budget_bytes,
                                 int64_t* cs);

/*
 * Bytes of device workspace dora_factored_norm needs for this shape.
 * The planner picks the most parallel split whose workspace fits
 * `budget_bytes`; the same arguments always give the same plan.
 * s == 0 or r == 0 needs no workspace (the cross and Gram terms are
 * skipped, cyqw.cn §5.1 notes). Host only; never touches the GPU.
 * Returns DORA_ERR_BUDGET if even the least parallel plan does not fit,
 * DORA_ERR_INVALID_ARG for negative sizes or ws_bytes == NULL,
 * DORA_ERR_UNSUPPORTED_DTYPE for an unknown dtype.
 */
dora_status dora_norm_workspace_size(int64_t d_out, int64_t d_in, int64_t r, int dtype,
                                     float s, size_t budget_bytes, size_t* ws_bytes);

/*
 * The plan dora_factored_norm would use, for diagnostics and benchmarks.
 * Fills info[0 .. n_info-1] with, in order: mode (0 nothing to do, 1 row
 * sum of squares only, 2 factored, 3 dense fused; in mode 3 the factored
 * fields describe the fallback used when the pointers do not allow aligned
 * 16-byte loads), W-pass column tile width, W-pass column
 * tiles, Gram-pass column tile width, Gram-pass column tiles, streaming and
 * general kernel configuration of the W pass, the same of the Gram pass,
 * d_in granule (elements), granules over d_in, d_in ranges of the W pass,
 * d_in ranges of the Gram pass, workspace bytes, W-pass grid and Gram-pass
 * grid of the streaming kernel, its LDS bytes in the W pass, the rows of
 * its W-pass tile, and 1 if the streaming W pass computes G itself (no
 * separate Gram pass; gram grid and ranges then do not apply), else 0,
 * 1 if the streaming Gram pass computes only the tiles on and above the
 * diagonal of G, else 0, and 1 if the streaming W pass also runs the Gram
 * term (B G) . B in its own accumulators (every dtype when G is not
 * folded in; no separate Gram-term pass), else 0, the index of the W
 * pass among the call's launches (see dora_factored_norm_marked), and 1 if
 * every operand tile of the streaming kernel spans less than 2^31 bytes
 * (its 32-bit buffer offsets; otherwise the general kernel runs), else 0,
 * and in mode 3 the dense pass's row tiles (64 rows) and column tiles (128
 * columns of d_in), else 0 and 0, and the d_in range groups of the
 * streaming W pass's die grid (the dies as range groups by row groups, so
 * that B's rows of a row tile are fetched by that many dies instead of one
 * die per range), 0 where it keeps the plain order; the streaming fields
 * apply when W, A and B allow aligned 16-byte loads.
 * Entries past the last field are set to -1.
 * Before returning it replays the plan on the host and checks that the
 * d_in ranges tile d_in exactly, every grid fits and every partial sum the
 * kernels write lies inside its workspace region; DORA_ERR_INVALID_ARG if
 * not. Host only; never touches the GPU.
 */
dora_status dora_norm_plan_info(int64_t d_out, int64_t d_in, int64_t r, int dtype, float s,
                                size_t budget_bytes, int64_t* info, int n_info);

/*
 * Factored row norm and magnitude scale (cyqw.cn §1.2, §1.2.1, §1.2.2,
 * §5.1 Algorithm 1; alanhou.org "Factored Norm").
 *
 *   wnorm[j] = sqrt(max(base[j] + 2s*cross[j] + s^2*ba[j], 0))
 *     base[j]  = sum_k W[j,k]^2
 *     cross[j] = sum_l B[j,l] * U[j,l],      U = W A^T   [d_out, r]
 *     ba[j]    = sum_l (B G)[j,l] * B[j,l],  G = A A^T   [r, r]
 *   g[j]     = m[j] / max(wnorm[j], eps)      (only if m != NULL)
 *
 * Inputs W, A, B are device pointers of storage type `dtype`; all
 * accumulation is fp32. U never leaves the matrix-core accumulators; BA is
 * never formed.
 *
 * Where r >= d_out, or r > d_in with d_out <= 4096 (bf16 and fp16, d_in
 * and r multiples of 8, plan mode 3), the Gram matrix or the Gram term
 * would cost more than B A itself, and the call computes the same wnorm
 * by its definition instead: a dense fused pass forms each 64 x 128 tile
 * of W + s B A in the matrix-core accumulators, squares it and keeps only
 * its row sums (cyqw.cn §1.1), and a second launch adds each row's tile
 * sums in a fixed order and takes the root. No tile of B A leaves the
 * chip; the workspace is the larger of the two paths' (the factored path
 * runs instead when W, A or B is not 16-byte aligned).
 *
 * wnorm (and g) are fp32 [d_out] device arrays written by the call. m is
 * an fp32 [d_out] device array or NULL (then g is not written and may be
 * NULL). A NaN in the inputs propagates to wnorm and g.
 *
 * `workspace` must hold at least dora_norm_workspace_size(...) bytes
 * (256-byte aligned) for the same (d_out, d_in, r, dtype, s, budget);
 * it may be NULL when that size is 0. Its contents on entry are ignored.
 *
 * Sizes may be 0: d_out == 0 does nothing; d_in == 0 gives wnorm = 0;
 * r == 0 or s == 0 gives wnorm = ||W||_row.
 *
 * Errors: DORA_ERR_INVALID_ARG (negative size, non-finite s or eps, eps <= 0,
 * required pointer NULL, output overlapping an input), DORA_ERR_UNSUPPORTED_DTYPE,
 * DORA_ERR_BUDGET (plan does not fit budget_bytes), DORA_ERR_WORKSPACE
 * (workspace_bytes too small or pointer misaligned), DORA_ERR_HIP.
 */
dora_status dora_factored_norm(const void* W, const void* A, const void* B, int dtype,
                               int64_t d_out, int64_t d_in, int64_t r, float s,
                               size_t budget_bytes, void* workspace, size_t workspace_bytes,
                               float* wnorm, const float* m, float eps, float* g,
                               void* stream);

/*
 * dora_factored_norm with timing marks: the same computation, arguments,
 * results and errors, and in addition HIP events recorded on `stream`
 * between the call's launches, so that a caller (a benchmark, a profiler)
 * can time each kernel of the norm on its own. events[0 .. n_events-1] are
 * hipEvent_t handles the caller created and owns; the call records
 * events[0] before its first launch and events[i] after its i-th launch,
 * for i < n_events (at most 8 are used); null entries are skipped (each
 * recorded event adds a little time between launches, so a caller that
 * times one launch passes only the two events around it). Nothing is kept
 * after the call returns. Launches of one call, in order:
 *   G not folded in: Gram pass, gram_reduce (fp16: which also splits B
 *     into bf16 hi + lo for the W pass), W pass with the Gram term (and
 *     the assembly when the W pass runs in one round of at most 256
 *     workgroups with at most 16 partials per row), assembly otherwise;
 *   G folded into the W pass (plan field gram_folded): W pass with G,
 *     gram_reduce, (fp16: widening of B,) Gram term (+ assembly with
 *     several Gram-term tiles);
 *   dense fused (plan mode 3): dense pass, assembly;
 *   s == 0, r == 0 or d_in == 0: one row-sum launch.
 * (These are the streaming-path launches, used when W, A and B allow
 * aligned 16-byte loads; plan field w_launch is the W pass's index i, which
 * lies between events[i] and events[i+1].)
 * Errors: those of dora_factored_norm, and DORA_ERR_INVALID_ARG for
 * n_events < 0 or events NULL with n_events > 0.
 */
dora_status dora_factored_norm_marked(const void* W, const void* A, const void* B, int dtype,
                                      int64_t d_out, int64_t d_in, int64_t r, float s,
                                      size_t budget_bytes, void* workspace, size_t workspace_bytes,
                                      float* wnorm, const float* m, float eps, float* g,
                                      void* stream, void* const* events, int n_events);

/*
 * Bytes of the device scratch array behind dora_factored_norm_noalloc: the
 * largest norm workspace that entry point can use (32 MiB per GPU).
 */
#define DORA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * dora_factored_norm for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same computation, arguments, results and errors, except
 * that there is no workspace argument. The workspace is a library-owned
 * array of DORA_NOALLOC_SCRATCH_BYTES in device memory, one per GPU, held
 * until the process ends; the call allocates nothing (no hipMalloc, no
 * library allocator). The plan is made under min(budget_bytes,
 * DORA_NOALLOC_SCRATCH_BYTES); a shape whose least parallel plan needs more
 * returns DORA_ERR_BUDGET before anything is enqueued. With the same plan
 * the results are bitwise those of dora_factored_norm. The scratch keeps
 * the last call's partial sums; every call overwrites what it reads, so
 * nothing needs clearing between calls. All calls on one GPU share its
 * scratch: calls that overlap in time on one GPU (on different streams, or
 * from different threads without ordering) race and give wrong results;
 * order them, e.g. on one stream. The first call on each GPU looks up the
 * array's device address (hipGetSymbolAddress, that GPU current); later
 * calls reuse it.
 */
dora_status dora_factored_norm_noalloc(const void* W, const void* A, const void* B, int dtype,
                                       int64_t d_out, int64_t d_in, int64_t r, float s,
                                       size_t budget_bytes, float* wnorm, const float* m, float eps,
                                       float* g, void* stream);

/*
 * g[j] = m[j] / max(wnorm[j], eps), fp32, on the device (cyqw.cn §1.2.2:
 * the magnitude division is kept apart from the fused kernels). A NaN
 * wnorm gives a NaN g. g may alias m or wnorm exactly.
 * Errors: DORA_ERR_INVALID_ARG (NULL pointer with d_out > 0, negative
 * d_out, eps not finite or <= 0), DORA_ERR_HIP.
 */
dora_status dora_magnitude_scale(const float* m, const float* wnorm, float eps,
                                 int64_t d_out, float* g, void* stream);

/*
 * out[j] = wnorm[j] rounded to the storage type `dtype` (round to nearest
 * even; DORA_F32 copies): the cast with which Algorithm 1 returns the norm
 * (cyqw.cn §5.1, step 7). dora_factored_norm keeps wnorm and g in fp32;
 * callers that want the pages' input-dtype norm apply this to its wnorm.
 * wnorm: fp32 [n] device array; out: [n] device array of `dtype`, owned by
 * the caller, not overlapping wnorm. Asynchronous on `stream`.
 * Errors: DORA_ERR_INVALID_ARG (negative n, NULL pointer with n > 0,
 * misaligned or overlapping pointers), DORA_ERR_UNSUPPORTED_DTYPE,
 * DORA_ERR_HIP.
 */
dora_status dora_norm_to_dtype(const float* wnorm, int64_t n, int dtype, void* out, void* stream);

/*
 * Stable magnitude compose (cyqw.cn §2.1, §2.1.1, §5.2):
 *
 *   out[t,j] = (g[j] - 1) * base[t,j] + g[j] * (s * lora[t,j])
 *
 * base, lora and out are [T, d_out] device arrays of storage type `dtype`;
 * g is an fp32 [d_out] device array. Arithmetic is fp32: s*lora is formed
 * first, then one fused multiply-add g*(s*lora) + (g-1)*base, rounded once
 * to the output type (round-to-nearest-even). One pass: base, lora and g
 * are read once and out is written once.
 * The result is the delta the DoRA layer adds to its base output.
 *
 * out may alias base or lora exactly (in-place); partial overlap is
 * rejected. T == 0 or d_out == 0 does nothing.
 * Errors: DORA_ERR_INVALID_ARG (NULL pointer with T*d_out > 0, negative
 * size, non-finite s, partial overlap), DORA_ERR_UNSUPPORTED_DTYPE,
 * DORA_ERR_HIP.
 */
dora_status dora_compose(const void* base, const void* lora, const float* g, float s,
                         int dtype, int64_t T, int64_t d_out, void* out, void* stream);

/*
 * DoRA layer output: the compose delta added to the base projection
 * (cyqw.cn §2.1.1: the layer returns base + delta; "Scaling DoRA",
 * alanhou.org, "The Problem": the adapted weight is m * V / ||V||_row with
 * V = W + sBA, so y = x V'^T = g * (base + s * lora) with base = x W^T,
 * lora = x A^T B^T):
 *
 *   y[t,j] = base[t,j] + ((g[j] - 1) * base[t,j] + g[j] * (s * lora[t,j]))
 *
 * Same arguments, layout, ownership and errors as dora_compose, with y in
 * place of out. The delta is formed in fp32 exactly as dora_compose forms
 * it, base is added in fp32, and y is rounded once to the storage type, in
 * the same single pass (base and lora read once, y written once).
 */
dora_status dora_layer_output(const void* base, const void* lora, const float* g, float s,
                              int dtype, int64_t T, int64_t d_out, void* y, void* stream);

/*
 * Workspace bytes dora_compose_backward needs to produce dg for a [T, d_out]
 * problem (at most 256 * d_out * 4). Host only. DORA_ERR_INVALID_ARG for
 * negative sizes or ws_bytes == NULL.
 */
dora_status dora_compose_backward_workspace_size(int64_t T, int64_t d_out, size_t* ws_bytes);

/*
 * Backward of the stable compose (cyqw.cn §4.2, §5.2, §6.1 Table 9 report
 * this fused backward; its formulas are the plain derivative of
 * delta = (g - 1) * base + g * (s * lora) with the row norm detached):
 *
 *   d_base[t,j] = (g[j] - 1) * dy[t,j]               (fp32, RNE to dtype)
 *   d_lora[t,j] = g[j] * (s * dy[t,j])               (fp32, RNE to dtype)
 *   dg[j]       = sum_t dy[t,j] * (base[t,j] + s * lora[t,j])     (fp32)
 *   dm[j]       = dg[j] / max(wnorm[j], eps)   (g = m / max(wnorm, eps))
 *
 * dy, base, lora, d_base, d_lora: device [T, d_out] row-major of `dtype`.
 * g, wnorm, dg, dm: fp32 [d_out] device arrays. Any of d_base, d_lora, dg
 * may be NULL to skip that output; with dg == NULL (magnitude frozen) base
 * and lora are not read and may be NULL. dm requires dg, wnorm and eps > 0.
 * dg is summed in fp32 in a fixed order (each thread's rows in increasing
 * order, then row blocks in increasing order): reproducible for a fixed
 * shape, no atomics. Outputs overlap no input and no other output.
 * `workspace` (256-byte aligned, dora_compose_backward_workspace_size bytes)
 * is needed only when dg != NULL; its contents on entry are ignored.
 * Asynchronous on `stream`.
 *
 * Errors: DORA_ERR_INVALID_ARG (negative size, non-finite s, bad eps,
 * missing or misaligned pointer, overlapping buffers),
 * DORA_ERR_UNSUPPORTED_DTYPE, DORA_ERR_WORKSPACE, DORA_ERR_HIP.
 */
dora_status dora_compose_backward(const void* dy, const void* base, const void* lora, const float* g,
                                  float s, int dtype, int64_t T, int64_t d_out, void* d_base,
                                  void* d_lora, float* dg, const float* wnorm, float eps, float* dm,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* -------------------------------------------------------------------------
 * The block around the adapted layer: the norm before it, and the product
 * with what surrounds it. Per-row and per-column vectors are fp32, like
 * wnorm, m and g above.
 * ---------------------------------------------------------------------- */

/*
 * Root-mean-square norm with the residual's addition:
 *
 *   h = x + residual
 *   rstd[t] = 1 / sqrt(mean_j h[t,j]^2 + eps)
 *   n[t,j]  = h[t,j] * rstd[t] * weight[j]
 *   y = n in the storage type;  scale[t] = max_j |n[t,j]| / 448 and
 *   q = n / scale[t] (the fp32 quotient) in e4m3 (both round to nearest even)
 *
 * x, residual, h, y: [T, d] of `dtype`; q: [T, d] bytes; weight: fp32 [d] or
 * NULL (ones); scale, rstd: fp32 [T]. residual NULL: h is x, and the h
 * argument must be NULL. h (with a residual), y, q and rstd may each be NULL
 * to skip them, but not y and q both; scale comes with q. h may be x or
 * residual itself. One launch, each input read once from memory (rows of
 * more than 16384 elements are read again).
 *
 * Arithmetic is fp32: the norm is of the unrounded sum x + residual, and h is
 * that sum rounded. A row of zeros has scale 1; a row whose largest |n| is
 * below 448 * 2^-100 has scale 2^-100. A NaN in a row makes its rstd, n,
 * scale and q NaN; an infinity (or a sum of squares past fp32's range) makes
 * rstd 0, so that n is 0, or NaN at the infinity, and scale and q are then
 * NaN as well. T == 0 does nothing; d == 0 has no norm and is refused when
 * scale or rstd is asked for. T and d are below 2^31, T * d at most 2^33.
 * Errors: DORA_ERR_INVALID_ARG (sizes, eps not finite or <= 0, missing,
 * misaligned or overlapping pointers), DORA_ERR_UNSUPPORTED_DTYPE,
 * DORA_ERR_HIP.
 */
dora_status dora_rms_norm(const void* x, const void* residual, const float* weight, float eps, int dtype, int64_t T,
                          int64_t d, void* h, void* y, void* q, float* scale, float* rstd, void* stream);

/*
 * Workspace bytes dora_rms_norm_backward needs for dweight. Host only.
 */
dora_status dora_rms_norm_backward_workspace_size(int64_t T, int64_t d, int dtype, size_t* ws_bytes);

/*
 * Backward of the norm, from the h and rstd of the forward (h is x where
 * there is no residual), with nh = h * rstd and a = dy * weight:
 *
 *   dx[t,j]    = rstd[t] * (a[t,j] - nh[t,j] * mean_j(a[t,:] nh[t,:])) + dh[t,j]
 *   dweight[j] = sum_t dy[t,j] * nh[t,j]
 *
 * dx is the gradient of x and of residual alike; dh is the gradient that
 * reaches h directly (the residual stream), or NULL. dx may be dy or dh
 * itself. dweight may be NULL (the weight frozen); it is summed in fp32 in a
 * fixed order, and needs the workspace (256-byte aligned).
 * Errors: as dora_rms_norm, and DORA_ERR_WORKSPACE.
 */
dora_status dora_rms_norm_backward(const void* dy, const void* dh, const void* h, const float* rstd,
                                   const float* weight, int dtype, int64_t T, int64_t d, void* dx, float* dweight,
                                   void* workspace, size_t workspace_bytes, void* stream);

typedef enum dora_act {
  DORA_ACT_NONE = 0,
  DORA_ACT_RELU = 1,
  DORA_ACT_GELU = 2,      /* z * Phi(z), by the error function              */
  DORA_ACT_GELU_TANH = 3, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))  */
  DORA_ACT_SILU = 4       /* z / (1 + exp(-z))                              */
} dora_act;

/*
 * Device workspace dora_matmul needs. `aligned_operands` has a bit for each
 * operand that starts on a 16-byte boundary (1 x, 2 w, 4 t, 8 b): an operand
 * that does not, or whose row length is no multiple of 16 bytes, is copied
 * into the workspace at a row stride that is. Host only.
 */
dora_status dora_matmul_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int aligned_operands,
                                       size_t* ws_bytes);

/*
 * The plan dora_matmul would use, for diagnostics and tests: info[0 ..
 * n_info-1] are, in order, the rows of its tile (256, 128 or 64; 0: the
 * kernel for few rows and small products; -1: nothing to do), the parts the
 * depth is split into (more than one are added by a second launch), a bit for
 * each operand that is copied first (as in dora_matmul_workspace_size), the
 * workspace bytes, and the rows that a workgroup of the few-rows kernel takes
 * (8, 16 or 32; -1 for a tile); further entries are -1. Host only.
 */
dora_status dora_matmul_plan_info(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int aligned_operands,
                                  int64_t* info, int n_info);

/*
 * Matrix product with its epilogue:
 *
 *   u[m,n] = row_scale[m] * (sum_k x[m,k] w[n,k] + s * sum_l t[m,l] b[n,l])
 *   y[m,n] = act(col_scale[n] * u[m,n] + bias[n]) + residual[m,n]
 *
 * x [M, K], w [N, K] of `dtype` (bf16, fp16, fp32 or DORA_E4M3); t [M, r] and
 * b [N, r] of the same type (the low-rank pair: t = x A^T, b = B; none with
 * r == 0, and none in e4m3). row_scale fp32 [M], col_scale and bias fp32 [N],
 * residual [M, N], each or NULL. y, u and residual are of `out_dtype`, which
 * is `dtype` except for e4m3 (any of the three). u, if not NULL, receives the
 * product before the column scale, for the backward (with a row_scale:
 * dora_matmul_backward_rows). y may be residual itself.
 *
 * With w = W, b = B, s the adapter's and col_scale = g of dora_factored_norm,
 * y is the whole DoRA layer g * (x W^T + s t B^T) + bias in one launch, with
 * neither projection written to memory. With e4m3 rows and scales of
 * dora_rms_norm as x and row_scale, col_scale carries the weight rows' scales.
 *
 * Products accumulate in fp32 on the matrix cores, the epilogue is fp32, and
 * y and u are each rounded once. The 8-bit matrix instructions align each
 * group of eight products to the largest of them and drop what lies 2^-13
 * below it: an e4m3 sum is off by up to 7 * 2^-13 of the sum of its products'
 * sizes more (about 2^-17 of it on normal data). Activations are accurate
 * relative to their value, in the tails too: an fp32 result to (16 + 2 z^2)
 * 2^-24 for gelu and (8 + 4 |e|) 2^-24 for the others, e being the argument of
 * their exponential; 16-bit results far below half a step. What is below
 * 2^-122 may be 0.
 *
 * `workspace` (256-byte aligned) holds at least dora_matmul_workspace_size
 * bytes; its contents on entry are ignored.
 * K == 0 gives u = s t b^T (0 without a pair); M == 0 or N == 0 does nothing.
 * Rows of x, w, t, b take less than 2^23 bytes, N is less than 2^23, M less
 * than 2^30, and no matrix has more than 2^33 elements.
 * Errors: DORA_ERR_INVALID_ARG (sizes, s not finite, unknown act, a pair in
 * e4m3, missing, misaligned or overlapping pointers),
 * DORA_ERR_UNSUPPORTED_DTYPE, DORA_ERR_WORKSPACE, DORA_ERR_HIP.
 */
dora_status dora_matmul(const void* x, const void* w, int dtype, int64_t M, int64_t N, int64_t K,
                        const float* row_scale, const float* col_scale, const void* t, const void* b, int64_t r,
                        float s, const float* bias, int act, const void* residual, int out_dtype, void* y, void* u,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Outputs of dora_matmul_backward, as its workspace query names them. */
#define DORA_GRAD_DX 1   /* dx                                  */
#define DORA_GRAD_DW 2   /* dw                                  */
#define DORA_GRAD_SUMS 4 /* dbias or dcol_scale, or both        */
#define DORA_GRAD_DU 8   /* du, in an array aligned to 16 bytes */
#define DORA_GRAD_ALIGNED 16 /* x (for dw) and w (for dx) start on 16-byte boundaries */

/* Device workspace dora_matmul_backward needs for a set of outputs. Host only. */
dora_status dora_matmul_backward_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                size_t* ws_bytes);

/*
 * Backward of a product without row_scale (bf16, fp16 or fp32), from the u of
 * the forward; the residual's gradient is dy itself:
 *
 *   z = col_scale[n] * u + bias[n]     dz = dy * act'(z)
 *   dbias[n] = sum_m dz                dcol_scale[n] = sum_m dz * u
 *   du = col_scale[n] * dz, rounded to the storage type
 *   dx = du w                          dw = du^T x
 *
 * dy, u, du [M, N]; dx [M, K]; dw [N, K]; dbias, dcol_scale fp32 [N]; any
 * output may be NULL. du may be dy itself. The low-rank pair's gradients are
 * those of two more products: with du as dy, act none and col_scale NULL,
 * x = t and w = b give s^-1 dt (dx) and s^-1 db (dw). Sums are fp32 in a
 * fixed order, without atomics; act' of relu at 0 is 0.
 * Errors: as dora_matmul; M and N too are limited to rows of less than 2^23
 * bytes.
 */
dora_status dora_matmul_backward(const void* dy, const void* u, const void* x, const void* w, int dtype, int64_t M,
                                 int64_t N, int64_t K, const float* col_scale, const float* bias, int act, void* du,
                                 void* dx, void* dw, float* dbias, float* dcol_scale, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * The same of a product with row_scale, fp32 [M] or NULL. u holds it, so z,
 * dz, dbias and dcol_scale are as above, and du is the gradient of the sum
 * that the row scale multiplies:
 *
 *   du = row_scale[m] * col_scale[n] * dz, rounded to the storage type
 *   dx = du w                          dw = du^T x
 *
 * The pair's gradients follow from this du by dora_matmul_backward, as above.
 * row_scale itself has no gradient here. Same workspace and errors.
 */
dora_status dora_matmul_backward_rows(const void* dy, const void* u, const void* x, const void* w, int dtype,
                                      int64_t M, int64_t N, int64_t K, const float* row_scale, const float* col_scale,
                                      const float* bias, int act, void* du, void* dx, void* dw, float* dbias,
                                      float* dcol_scale, void* workspace, size_t workspace_bytes, void* stream);

/* -------------------------------------------------------------------------
 * Rows held in 8-bit integers: int8 values, each the nearest step of its
 * scale, and fp32 scales, one a row or one for each group of columns of a
 * row. The layer norm and dora_quantize_rows write them, dora_matmul_int8
 * multiplies them, dora_matmul_backward_int8 reads them as checkpoints.
 *
 *   scale = max |x| / 127      q = x / scale to the nearest integer, ties to
 *                              the even one
 *
 * with the maximum over the row or the group. The scale is the quotient
 * rounded once to fp32; q is that of the exact quotient by the scale so held.
 * Zeros have scale 1; a scale is at least 2^-100. A NaN or an infinity makes
 * the scale NaN or infinite and q 0, so that every value of that row or group
 * stands for NaN.
 * ---------------------------------------------------------------------- */

/* 8-bit integers, where an output's 8-bit type is chosen. */
#define DORA_I8 4

/*
 * Layer norm with the residual's addition:
 *
 *   h = x + residual
 *   mean[t] = mean_j h[t,j]
 *   rstd[t] = 1 / sqrt(mean_j (h[t,j] - mean[t])^2 + eps)
 *   n[t,j]  = (h[t,j] - mean[t]) * rstd[t] * weight[j] + bias[j]
 *   y = n in the storage type
 *   q, scale: n in 8 bits, by q_dtype DORA_E4M3 (scale = max_j |n| / 448, as
 *   dora_rms_norm) or DORA_I8 (above)
 *
 * Arguments as dora_rms_norm, and bias: fp32 [d] or NULL (zeros); mean: fp32
 * [T] or NULL. h (with a residual), y, q, mean and rstd may each be NULL to
 * skip them, but not y and q both; scale comes with q. y and q may be written
 * together. h may be x or residual itself. One launch, each input read once
 * from memory (rows of more than 16384 elements are read again).
 *
 * The statistics are of the unrounded fp32 sum, the variance of the values
 * about their mean. A NaN or an infinity in a row (or a sum of its values or
 * of their squares about the mean past fp32's range) makes its mean, rstd, n
 * and scale NaN. T == 0 does nothing; d == 0 has no norm and is refused when
 * scale, mean or rstd is asked for. T and d are below 2^31, T * d at most 2^33.
 * Errors: as dora_rms_norm; an unknown q_dtype with q is
 * DORA_ERR_UNSUPPORTED_DTYPE.
 */
dora_status dora_layer_norm(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                            int dtype, int64_t T, int64_t d, void* h, void* y, void* q, int q_dtype, float* scale,
                            float* mean, float* rstd, void* stream);

/* Workspace bytes dora_layer_norm_backward needs for dweight or dbias. Host only. */
dora_status dora_layer_norm_backward_workspace_size(int64_t T, int64_t d, int dtype, size_t* ws_bytes);

/*
 * Backward of the layer norm, from the h, mean and rstd of the forward (h is x
 * where there is no residual), with nh = (h - mean) * rstd and a = dy * weight:
 *
 *   dx[t,j]    = rstd[t] * (a[t,j] - mean_j(a[t,:]) - nh[t,j] * mean_j(a[t,:] nh[t,:])) + dh[t,j]
 *   dweight[j] = sum_t dy[t,j] * nh[t,j]        dbias[j] = sum_t dy[t,j]
 *
 * dx is the gradient of x and of residual alike; dh is the gradient that
 * reaches h directly, or NULL. dx may be dy or dh itself. dweight and dbias
 * may each be NULL; they are summed in fp32 in a fixed order, and need the
 * workspace (256-byte aligned).
 * Errors: as dora_layer_norm, and DORA_ERR_WORKSPACE.
 */
dora_status dora_layer_norm_backward(const void* dy, const void* dh, const void* h, const float* mean,
                                     const float* rstd, const float* weight, int dtype, int64_t T, int64_t d, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * x [T, d] of `dtype` to int8 rows: q int8 [T, d], and scale fp32 [T] (group
 * 0: one a row) or [T, ceil(d / group)] (group 32, 64, 128 or 256 columns, the
 * last group what is left). One launch. T == 0 does nothing, and so does
 * d == 0 with groups; without them it is refused.
 * Errors: DORA_ERR_INVALID_ARG (sizes, group, missing, misaligned or
 * overlapping pointers), DORA_ERR_UNSUPPORTED_DTYPE, DORA_ERR_HIP.
 */
dora_status dora_quantize_rows(const void* x, int dtype, int64_t T, int64_t d, int64_t group, int8_t* q, float* scale,
                               void* stream);

/* x = q * scale, rounded once to `dtype`: the values that int8 rows stand for. Arguments and errors alike. */
dora_status dora_dequantize_rows(const int8_t* q, const float* scale, int64_t T, int64_t d, int64_t group, int dtype,
                                 void* x, void* stream);

/*
 * Workspace and plan of dora_matmul_int8, as those of dora_matmul (x and w are
 * int8, t and b of 16 bits), but that small products, and products of up to 64
 * rows as to w, read operands off the 16-byte grid as they are (K and r of
 * less than 16 bytes apart). The workspace for operands at any address
 * (aligned_operands 0) serves them at all. The plan's sixth entry names the
 * kernel: 0 tiles whose operands lie on the grid, 1 few rows, 2 few rows with
 * the tokens in registers, which walks the columns, 3 tiles of 64 rows whose
 * operands lie at any address (-1: nothing to do). Host only.
 */
dora_status dora_matmul_int8_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int aligned_operands,
                                            size_t* ws_bytes);
dora_status dora_matmul_int8_plan_info(int64_t M, int64_t N, int64_t K, int64_t r, int aligned_operands, int64_t* info,
                                       int n_info);

/*
 * Matrix product in 8-bit integers with a scale for each token and channel:
 *
 *   u[m,n] = row_scale[m] * w_scale[n] * sum_k x[m,k] w[n,k] + s * sum_l t[m,l] b[n,l]
 *   y[m,n] = act(col_scale[n] * u[m,n] + bias[n]) + residual[m,n]
 *
 * x int8 [M, K] with row_scale fp32 [M], w int8 [N, K] with w_scale fp32 [N]:
 * int8 rows with one scale a row (any int8 value is taken, -128 too). y, u and
 * residual are of `out_dtype` (bf16, fp16 or fp32); t [M, r] and b [N, r], the
 * low-rank pair, are of `out_dtype`, bf16 or fp16 (none with r == 0, and none
 * with fp32 outputs). With w an int8 copy of the frozen W, b = B, s the
 * adapter's and col_scale = g, y is the whole DoRA layer on an 8-bit base. The
 * other arguments are those of dora_matmul, and y may be residual itself.
 *
 * The sum over k is exact in int32 (K is at most 131071); it is converted to
 * fp32 and multiplied by the scales there (parts of a split depth, and the
 * eighths of a few rows' depth, each by themselves). With a pair that sum is
 * divided by s and multiplied again, so |s| is between 2^-64 and 2^64, or s is
 * 0 and the pair is not read.
 * Errors: as dora_matmul, and DORA_ERR_INVALID_ARG for K past its limit, such
 * an s, and a pair with fp32 outputs.
 */
dora_status dora_matmul_int8(const int8_t* x, const float* row_scale, const int8_t* w, const float* w_scale, int64_t M,
                             int64_t N, int64_t K, const float* col_scale, const void* t, const void* b, int64_t r,
                             float s, const float* bias, int act, const void* residual, int out_dtype, void* y, void* u,
                             void* workspace, size_t workspace_bytes, void* stream);

/* An operand held as int8 rows: scale [rows] with group 0, else [rows, ceil(columns / group)]. */
typedef struct dora_int8_rows {
  const int8_t* q;
  const float* scale;
  int64_t group;
} dora_int8_rows;

/* Operands of dora_matmul_backward_int8 held as int8 rows, as its workspace query names them. */
#define DORA_HELD_X 1
#define DORA_HELD_W 2

/*
 * Device workspace dora_matmul_backward_int8 needs: `outputs` as for
 * dora_matmul_backward (DORA_GRAD_ALIGNED speaks of x, or x8's q, and of w, or
 * w8's q), `held` the DORA_HELD_ bits. Rows of several scales may need less
 * than this: the second query, with how many scales a row of x8 and of w8 has
 * (0: x or w is not held so), says how much. Host only.
 */
dora_status dora_matmul_backward_int8_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs, int held,
                                                     size_t* ws_bytes);
dora_status dora_matmul_backward_int8_scales_workspace_size(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                            int64_t x_scales, int64_t w_scales, size_t* ws_bytes);

/*
 * The plan it would use, for diagnostics and tests: info[0 .. n_info-1] are, of
 * dx and then of dw, the rows of the product's tile (0: the kernel for few rows
 * and small products), the parts of its depth, and how it reads w (dx) or x
 * (dw): 0 as it lies, 1 from a copy (of int8 rows in 16 bits, at whole chunks,
 * transposed in fp32), 2 as the int8 rows that are held (-1 for a gradient that
 * is not asked for or empty); then the workspace bytes; further entries are -1.
 * Host only.
 */
dora_status dora_matmul_backward_int8_plan_info(int64_t M, int64_t N, int64_t K, int dtype, int outputs,
                                                int64_t x_scales, int64_t w_scales, int64_t* info, int n_info);

/*
 * dora_matmul_backward_rows with any of u, x and w held as int8 rows: u8, x8
 * and w8 stand in for u, x and w, of which each is given in one of the two
 * forms (the other NULL). u8 [M, N] and x8 [M, K] are activations packed in
 * the forward; w8 [N, K] is a frozen 8-bit base (the gradient dw of such a w,
 * if asked for, is that of the values it stands for).
 *
 *   z = col_scale[n] * u + bias[n]   with u = u8.q * its scale in fp32
 *   dx = du (w8.q * its scale)       dw = du^T (x8.q * its scale)
 *
 * The products' operands are of the storage type, so the values of x8 and w8
 * are rounded to it, as du is. Those of rows with one scale are not: in 16 bits
 * such a product's other operand is du times the scale's significand, rounded
 * once, and the integers times the scale's power of two are exact. And of x8 in
 * groups with act none and no row_scale dw is col_scale times dy^T x, without
 * du's rounding, where dy lies on a 16-byte boundary (and is not du), and N is a
 * multiple of 8. Everything else, the workspace and the errors are as there.
 */
dora_status dora_matmul_backward_int8(const void* dy, const void* u, const dora_int8_rows* u8, const void* x,
                                      const dora_int8_rows* x8, const void* w, const dora_int8_rows* w8, int dtype,
                                      int64_t M, int64_t N, int64_t K, const float* row_scale, const float* col_scale,
                                      const float* bias, int act, void* du, void* dx, void* dw, float* dbias,
                                      float* dcol_scale, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DORA_H_ */
