/*
 * himuon.h - C ABI of the MI355X (gfx950) tiled Newton-Schulz library.
 *
 * What the library computes
 * -------------------------
 * HiMuon ("Hierarchical Muon: Tiled Newton-Schulz Updates for Efficient Muon
 * Optimization", arXiv 2606.27216, abstract): every H x W momentum matrix is
 * cut into T x T tiles anchored at (0, 0) (the last tile row and column hold
 * the remainder, processed at their own h x w size), the same finite
 * Newton-Schulz map is applied to every tile independently, and the results
 * are written back in place.
 *
 * The per-tile map is Algorithm 1 of the "Gram Newton-Schulz" summary page
 * (section 3, standard Newton-Schulz): X = Y / (||Y||_F + eps), then for
 * t = 1..K:  A = X X^T,  B = b_t A + c_t A^2,  X = a_t X + B X.
 * (The page's transpose of tall blocks only changes the cost: each step is an
 * odd matrix polynomial, so the result is the same either way.)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Matrices are row-major in device memory: element (i, j) of a descriptor
 *   sits at ptr + i * ld + j (in elements).  rows >= 1, cols >= 1, ld >= cols.
 *   All matrices of one call share one dtype.  Pointers must be aligned to the
 *   element size; no other alignment is required (16-byte aligned rows take a
 *   vector fast path).
 * - The caller owns all device memory.  The library allocates no device memory
 *   and keeps no device state between calls (himuon_tiled_ns_noalloc aside,
 *   which uses a fixed scratch array the library holds on each device).  The descriptor array and the
 *   coefficient array are read during the call only.  A call issues kernel
 *   launches only (no memsets or copies), so it may be captured in a HIP graph,
 *   and calls on different streams may run at once on disjoint matrices and
 *   workspaces.
 * - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream) and
 *   the call returns without waiting.  Results are valid once the stream has
 *   reached that point.  The workspace must stay allocated until then.
 * - Validation is all-or-nothing: when a call returns anything but HIMUON_OK,
 *   nothing was enqueued and no memory was touched (HIMUON_ERR_HIP excepted: it
 *   reports a launch failure from the HIP runtime; himuon_last_hip_error()
 *   returns the hipError_t).
 * - Matrices of one call must not overlap in memory (they are written in
 *   place).  No exception crosses this interface.
 * - Non-finite inputs are not an error: a NaN or Inf stays inside its tile.
 * - bf16 tiles with both sides from 48 to 256 or from 32 to 128 (and tiles
 *   with both sides at most 64) stay resident on chip for all K steps and
 *   need no workspace: one kernel launch per group of up to 256 tile classes (a class
 *   is one matrix's interior, right-edge, bottom-edge or corner tiles), plus
 *   one for a partly filled last round of 128-tiles.  fp32 tiles with both
 *   sides at most 64 stay on chip too (fp32 MFMA, one launch per group).
 *   Larger tiles, thin tiles, larger fp32 tiles, and the full-matrix map
 *   (T >= max(rows, cols)) run step by step through the caller's workspace,
 *   in chunks of tiles that each fit in `workspace_bytes`; that workspace is
 *   bf16 for bf16 tiles whose sides are both at least 64, fp32 otherwise.
 *   HIMUON_BF16_PRECISE runs every tile on the step-by-step path with an
 *   fp32 workspace.
 */
#ifndef HIMUON_H
#define HIMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Largest K accepted by any entry point. */
#define HIMUON_MAX_STEPS 16

/* One matrix: device pointer to element (0, 0), its size and row stride. */
typedef struct himuon_matrix {
    void*   ptr;   /* device pointer, aligned to the element size           */
    int64_t rows;  /* H >= 1                                                 */
    int64_t cols;  /* W >= 1                                                 */
    int64_t ld;    /* row stride in elements, ld >= cols                     */
} himuon_matrix_t;

/*
 * Storage and arithmetic.  The pages cast the normalised block to bf16 and
 * leave later precision open ("Gram Newton-Schulz" page, section 3,
 * Algorithm 1; section 6 notes on low-precision Gram iterations).
 *
 * Accuracy contract: the error of a tile is ||out - ref||_F / ||ref||_F with
 * ref the exact (fp64) map of the stored input; the bound is on the worst tile.
 *  - HIMUON_FP32: <= 1e-4 (measured at most a few 1e-6).
 *  - HIMUON_BF16: <= 3e-2 (measured 1.1e-2 to 2.0e-2 on the worst of 10^4 to
 *    10^6 random full-rank tiles per kernel size) for
 *      * K <= 5 steps (the quintic (3.4445, -4.7750, 2.0315) every step, or
 *        per-step mixes with cubic steps); tiles of up to 32 also for longer
 *        runs of converging steps, such as five quintic then eleven cubic
 *        (1.5, -0.5, 0) steps, which larger tiles exceed on a tail of tiles
 *        (1-3 % of random tiles, worst 0.15-0.25);
 *      * tiles without near-zero singular values (relative to the largest);
 *      * entries of magnitude about 1e-15 to 1e15 (tested at 2^-50 and
 *        2^50, with eps scaled to the data): the Frobenius reduction, and at
 *        kernel tile 128 the product X X^T of the raw tile, run in fp32 and
 *        underflow below about 1e-18 or overflow above about 1e17.
 *    It does NOT hold for tiles of low numerical rank (rank 1 to 16 of a
 *    128-tile: 0.17-0.29 measured), because the iterate is rounded to bf16
 *    every step and each step multiplies its small singular values by about
 *    a_t; nor for 16 quintic steps in a row (0.04-0.18 measured, by kernel
 *    size; the quintic keeps singular values where its slope exceeds 1, so
 *    every rounding grows from step to step).
 *  - HIMUON_BF16_PRECISE: bf16 storage, fp32 arithmetic throughout (the
 *    fp32 step-by-step path, fp32 MFMA); the result is rounded to bf16 once.
 *    <= 3e-2 also on the cases above (measured 1.7e-3 to 2.0e-3, mostly the
 *    final rounding), at a much lower throughput.  For calls whose tiles may
 *    be of low rank or that run many quintic steps.
 */
typedef enum himuon_dtype {
    HIMUON_BF16 = 0,          /* bfloat16 storage; bf16 MFMA with fp32 accumulation */
    HIMUON_FP32 = 1,          /* float32 storage; fp32 arithmetic throughout        */
    HIMUON_BF16_PRECISE = 2   /* bfloat16 storage; fp32 arithmetic throughout       */
} himuon_dtype_t;

typedef enum himuon_status {
    HIMUON_OK = 0,
    HIMUON_ERR_INVALID_ARGUMENT = 1, /* null pointer, size < 1, ld < cols, K or eps out of range, non-finite coefficient */
    HIMUON_ERR_UNSUPPORTED = 2,      /* dtype or option the library does not provide                                  */
    HIMUON_ERR_LAYOUT = 3,           /* pointer not aligned to the element size, or an index that overflows int64   */
    HIMUON_ERR_OVERLAP = 4,          /* two matrices that are written share memory                                  */
    HIMUON_ERR_WORKSPACE = 5,        /* workspace too small for one tile of the step-by-step path, or NULL with bytes > 0 */
    HIMUON_ERR_HIP = 6               /* the HIP runtime refused a launch                                            */
} himuon_status_t;

/* Summary of how a call would be carried out (host-side planning only). */
typedef struct himuon_plan_info {
    int64_t tiles;            /* tiles over all matrices                              */
    int64_t resident_launches;/* launch groups of the on-chip kernels (tiles <= 256, bf16) */
    int64_t chunks;           /* chunks of the step-by-step path (0 if not used)      */
    int64_t launches;         /* total kernel launches one call enqueues              */
    int64_t kernel_tile;      /* largest on-chip kernel size (32, 64, 128 or 256), or 0 */
    size_t  workspace_full;   /* bytes the step-by-step path needs for one chunk      */
    size_t  workspace_min;    /* bytes it needs for its largest single tile           */
    int64_t tail_tiles;       /* 128-tiles of the partial last round, run eight waves
                                 per tile by a second launch on the current device
                                 (0 when no device is visible)                        */
} himuon_plan_info_t;

/*
 * himuon_plan - describe how himuon_tiled_ns(m, n, T, K, ..., dt, ...,
 * workspace_bytes) would run, without touching the GPU.  workspace_bytes is
 * the cap the chunking must respect (ignored when no workspace is needed).
 * Returns the same validation status the call would return (pointers are not
 * dereferenced).
 */
himuon_status_t himuon_plan(const himuon_matrix_t* m, int32_t n, int32_t T, int32_t K,
                            himuon_dtype_t dt, size_t workspace_bytes,
                            himuon_plan_info_t* info);

/*
 * himuon_workspace_size - bytes of device workspace himuon_tiled_ns needs to
 * run all tiles of these matrices in a single chunk (*full) and the least it
 * accepts (*min, one tile).  Both are 0 when the call needs no workspace.
 * Either output pointer may be NULL.
 */
himuon_status_t himuon_workspace_size(const himuon_matrix_t* m, int32_t n, int32_t T,
                                      himuon_dtype_t dt, size_t* full, size_t* min);

/*
 * himuon_tiled_ns - HiMuon tiled Newton-Schulz, in place, on n matrices.
 *
 * m, n       : n >= 0 matrix descriptors (n == 0 is a no-op).
 * T          : tile edge, T >= 1.  Tiles are T x T anchored at (0, 0); edge
 *              tiles are h x w with h, w <= T.  T >= max(rows, cols) gives the
 *              full-matrix Newton-Schulz map of each matrix.
 * K          : number of Newton-Schulz steps, 0 <= K <= HIMUON_MAX_STEPS
 *              (K = 0 writes the Frobenius-normalised tiles).
 * abc        : 3*K floats, step t uses (a_t, b_t, c_t) = abc[3t .. 3t+2];
 *              may be NULL when K == 0.  Must be finite.
 * dt         : storage dtype of every matrix.
 * eps        : added to each tile's Frobenius norm (>= 0, finite); 1e-7 in
 *              the page's Algorithm 1.
 * workspace, workspace_bytes : device scratch for the step-by-step path; the
 *              tiles are processed in chunks that fit.  May be NULL / 0 when
 *              himuon_workspace_size reports 0.
 * stream     : hipStream_t to enqueue on.
 */
himuon_status_t himuon_tiled_ns(const himuon_matrix_t* m, int32_t n, int32_t T, int32_t K,
                                const float* abc, himuon_dtype_t dt, float eps,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device scratch the library holds for himuon_tiled_ns_noalloc. */
#define HIMUON_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)

/*
 * himuon_tiled_ns_noalloc - himuon_tiled_ns for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, and
 * harnesses that forbid hipMalloc.  It computes exactly what himuon_tiled_ns
 * computes (same kernels, same per-tile arithmetic, so the same bits) and
 * allocates nothing: the step-by-step path runs through a fixed scratch array
 * of HIMUON_NOALLOC_SCRATCH_BYTES (128 MiB) that the library holds on every
 * device it runs on, from the first use there until the process ends.  Tiles
 * are processed in chunks that fit it.
 *
 * Arguments as for himuon_tiled_ns, without the workspace.
 * Errors: as for himuon_tiled_ns; HIMUON_ERR_WORKSPACE when one tile of the
 * step-by-step path needs more than HIMUON_NOALLOC_SCRATCH_BYTES on its own
 * (for example a full-matrix map above about 64 M bf16 elements), reported
 * before the device is touched; HIMUON_ERR_HIP if the scratch address cannot
 * be obtained on the current device.
 * Every call on one device shares that device's scratch, which keeps the last
 * call's contents (nothing in it needs to start at zero).  Calls whose work
 * overlaps in time on one device (other streams, other threads) race on it:
 * order them on one stream, or use himuon_tiled_ns with separate workspaces.
 */
himuon_status_t himuon_tiled_ns_noalloc(const himuon_matrix_t* m, int32_t n, int32_t T, int32_t K,
                                        const float* abc, himuon_dtype_t dt, float eps, void* stream);

/*
 * himuon_tiled_ns_schedule - K Newton-Schulz steps with a tile size per step:
 * step k works on the T[k] x T[k] tiles (HiMuon abstract, "runtime tile-size
 * schedules", read as a per-step tile size).  Each tile of the first size is
 * normalised once (eps added to its Frobenius norm); later steps use the
 * tiles as they stand.  The sizes must not increase and each must divide the
 * one before, so a finer tile lies inside one coarser tile; the step count of
 * a size and its coefficients are taken in order from abc (3 K floats, host).
 * Steps of one size run as one himuon_tiled_ns pass; between passes the
 * matrices hold the current iterate in their own dtype.
 *
 * Arguments as for himuon_tiled_ns, with T a host array of K tile sizes.
 * workspace_bytes caps every pass; the workspace must fit the largest need of
 * any pass (himuon_workspace_size for that pass's tile size).
 * Errors: HIMUON_ERR_INVALID_ARGUMENT for K < 1 or > HIMUON_MAX_STEPS, a
 * null T, a size < 1, or sizes that increase or do not nest; otherwise as for
 * himuon_tiled_ns.  Every pass is validated before the first is enqueued.
 */
himuon_status_t himuon_tiled_ns_schedule(const himuon_matrix_t* m, int32_t n, const int32_t* T, int32_t K,
                                         const float* abc, himuon_dtype_t dt, float eps, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * himuon_muon_step - fused Muon update with the tiled map in place of polar()
 * ("Gram Newton-Schulz" summary page, section 3, the Muon update rule):
 *     M <- mu M + G            (stored back into M, rounded to dt)
 *     W <- W - eta * tiledNS(M)
 * W[i], M[i], G[i] must have equal rows and cols (their ld may differ).  W and
 * M are written; G is read only.  No W, M or G may overlap any written matrix.
 * Other arguments as for himuon_tiled_ns; mu and eta must be finite.
 */
himuon_status_t himuon_muon_step(const himuon_matrix_t* W, const himuon_matrix_t* M,
                                 const himuon_matrix_t* G, int32_t n, int32_t T, int32_t K,
                                 const float* abc, float mu, float eta, himuon_dtype_t dt,
                                 float eps, void* workspace, size_t workspace_bytes, void* stream);

/*
 * himuon_gram_ns - the full-matrix Newton-Schulz map of each matrix, in place,
 * computed through its Gram matrix ("Gram Newton-Schulz" summary page,
 * section 6, Algorithm 3, stabilised Gram Newton-Schulz with a restart).
 *
 * Each matrix Y is normalised, X = Y / (||Y||_F + eps), and oriented so that
 * X is r x s with r <= s (a tall matrix is worked on transposed).  The steps
 * then run on r x r matrices:
 *     R = X X^T,  Q = I;   for t = 1..K:
 *         P = a_t I + b_t R + c_t R^2,   Q <- P Q,   R <- P R P
 * and the result Q X is written back (in the matrix's own orientation).  In
 * exact arithmetic this equals himuon_tiled_ns with T >= max(rows, cols); the
 * iteration costs about 4 r^3 flops a step instead of 4 r^2 s + 2 r^3, so it
 * pays for wide matrices (s well above r).  Before step restart + 1 the
 * iteration restarts (the page restarts before its third step, restart = 2):
 * X <- Q X,  R <- X X^T,  Q <- I, which removes the rounding R has gathered.
 *
 * m, n       : n >= 0 matrix descriptors, as for himuon_tiled_ns.
 * K, abc     : steps and coefficients, as for himuon_tiled_ns.
 * restart    : >= 0; 0 (or >= K) never restarts (the page's Algorithm 2).
 * dt, eps    : as for himuon_tiled_ns.
 * workspace, workspace_bytes : device scratch, at least the *min of
 *              himuon_gram_ns_workspace; matrices are processed in chunks
 *              that fit (every matrix runs on the step-by-step path; K = 0
 *              writes the normalised matrices as himuon_tiled_ns does).
 * stream     : hipStream_t to enqueue on.
 * The workspace holds the iterates in bf16 when dt is bf16 and both sides of
 * the matrix are at least 96, else in fp32 (smaller Gram matrices lose too
 * much accuracy to bf16 rounding).
 * Errors: HIMUON_ERR_INVALID_ARGUMENT for restart < 0, otherwise as for
 * himuon_tiled_ns (HIMUON_ERR_LAYOUT also for a side above INT32_MAX).
 */
himuon_status_t himuon_gram_ns(const himuon_matrix_t* m, int32_t n, int32_t K, const float* abc,
                               int32_t restart, himuon_dtype_t dt, float eps, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Bytes of workspace himuon_gram_ns needs for these matrices in one chunk
 * (*full) and for its largest single matrix (*min).  Host-side only; either
 * output pointer may be NULL. */
himuon_status_t himuon_gram_ns_workspace(const himuon_matrix_t* m, int32_t n, himuon_dtype_t dt,
                                         size_t* full, size_t* min);

/*
 * himuon_pair_stats - for n pairs of equal-shaped matrices (a[i], b[i]) the
 * three sums  sum a*b,  sum a*a,  sum b*b  over all elements, in fp64.
 *
 * They measure how far a tiled Newton-Schulz output lies from the
 * full-matrix map of the same input (HiMuon abstract: the tiled map acts on
 * each tile alone, where the full map couples all rows and columns; the pages
 * give no measure of that gap).  With g = tiled, f = full:
 *     ||g - f||_F / ||f||_F = sqrt(gg + ff - 2 gf) / sqrt(ff),
 *     cosine = gf / sqrt(gg ff).
 *
 * a, b     : n descriptors each (host arrays, read during the call); a[i] and
 *            b[i] must have equal rows and cols (their ld may differ).  Read
 *            only; they may overlap each other.
 * dt       : element type of every matrix.
 * out      : device array of 3 n doubles, written (out[3i .. 3i+2] =
 *            sum a*b, sum a*a, sum b*b of pair i); 8-byte aligned.
 * workspace, workspace_bytes : device scratch for per-workgroup partial sums,
 *            at least himuon_pair_stats_workspace(a, n) bytes, 8-byte aligned.
 * stream   : hipStream_t to enqueue on.
 * Products are exact in fp64 and summed in fp64 in a fixed order: the same
 * inputs give the same bits on every run.
 * Errors: HIMUON_ERR_INVALID_ARGUMENT (null pointer, size < 1, ld < cols,
 * shapes that differ), HIMUON_ERR_UNSUPPORTED (dtype), HIMUON_ERR_LAYOUT
 * (misaligned pointer), HIMUON_ERR_WORKSPACE (workspace NULL or too small),
 * HIMUON_ERR_HIP (launch refused).  n == 0 is a no-op.
 */
himuon_status_t himuon_pair_stats(const himuon_matrix_t* a, const himuon_matrix_t* b, int32_t n,
                                  himuon_dtype_t dt, double* out, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Bytes of workspace himuon_pair_stats needs for pairs of these shapes (the
 * shapes of `a`; pointers are not read).  Host-side only. */
himuon_status_t himuon_pair_stats_workspace(const himuon_matrix_t* a, int32_t n, size_t* bytes);

/* ==========================================================================
 * Operators around the optimiser step
 *
 * The matrices this library orthogonalises are the weights of language
 * models.  The entry points below compute what such a training step needs
 * next to it: the products of a mixture-of-experts layer (whose weight
 * gradient is the G of himuon_muon_step), the loss of a student against a
 * teacher's top logits, and the log probabilities of given tokens.  The
 * conventions at the top of this file hold, with these additions:
 * - X, Y, D (rows of tokens) and logits may have 0 rows; their pointer may
 *   then be NULL.
 * - dt is HIMUON_BF16 or HIMUON_FP32 (HIMUON_ERR_UNSUPPORTED otherwise).
 *   bf16 products are accumulated in fp32 and rounded once; softmax
 *   statistics, losses and log probabilities are fp32 for either type.
 * - Arrays named as device arrays are contiguous and aligned to their
 *   element.  Their contents are not validated on the host; the kernels clamp
 *   or skip as stated, and never access memory outside the operands.  (An
 *   operand reaches from its first element to its last: what lies between its
 *   rows may be read, and is not used, but never written.)
 * - Results do not depend on scheduling: the same inputs give the same bits.
 * ========================================================================== */

/*
 * himuon_grouped_mm - matrix products grouped by expert with ragged sizes.
 *
 *     Y[r, :] = X[r, :] W_e      for every row r of expert e
 *
 * X        : M x K, rows sorted by expert.
 * W, n     : n >= 1 weight matrices, all of one shape: K x N, or N x K when
 *            trans_w is not 0 (then Y = X W_e^T; with the weights of a forward
 *            product and trans_w flipped this is its input gradient).
 * ends     : device array of n int32, non-decreasing: expert e owns rows
 *            [ends[e-1], ends[e]) with ends[-1] = 0.  An expert may own no
 *            row.  Values are clamped to [0, M]; rows at or past ends[n-1]
 *            belong to no expert and become zero.  (An array that decreases
 *            gives unspecified values in Y, but no access outside it.)
 * Y        : M x N, written; must not overlap X or any W.
 * stream   : hipStream_t to enqueue on.
 * One launch per 255 experts.  The fast paths are for bf16 operands of 16-byte
 * chunks: K and N multiples of 8, every matrix at a 16-byte aligned address with
 * a row stride that is a multiple of 8, at most 2^22.  Other bf16 operands are
 * multiplied at about half their rate.
 * Errors: HIMUON_ERR_INVALID_ARGUMENT (null pointer, n < 1, shapes that do not
 * match), HIMUON_ERR_UNSUPPORTED (dtype), HIMUON_ERR_LAYOUT (alignment, a side
 * above INT32_MAX - 4096, or more output tiles than a launch can hold),
 * HIMUON_ERR_OVERLAP, HIMUON_ERR_HIP.
 */
himuon_status_t himuon_grouped_mm(const himuon_matrix_t* X, const himuon_matrix_t* W, int32_t n, int32_t trans_w,
                                  const int32_t* ends, const himuon_matrix_t* Y, himuon_dtype_t dt, void* stream);

/*
 * himuon_grouped_wgrad - the weight gradients of himuon_grouped_mm.
 *
 *     G_e = X_e^T D_e,   X_e and D_e the rows of expert e
 *
 * X, D     : M x K and M x N, rows sorted by expert (D = dL/dY).
 * G, n     : n >= 1 matrices of K x N, written (zero for an expert without
 *            rows); they must not overlap each other, X or D.  For weights
 *            stored N x K, pass D as X and X as D.
 * ends     : as for himuon_grouped_mm; rows past ends[n-1] count nowhere.
 * workspace: device scratch of at least himuon_grouped_wgrad_workspace bytes,
 *            16-byte aligned; may be NULL when that is 0.  Where G is small and
 *            the rows are many, these are cut into parts whose sums are added in
 *            order.
 * Errors as for himuon_grouped_mm, and HIMUON_ERR_WORKSPACE.
 */
himuon_status_t himuon_grouped_wgrad(const himuon_matrix_t* X, const himuon_matrix_t* D, const int32_t* ends,
                                     const himuon_matrix_t* G, int32_t n, himuon_dtype_t dt, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Bytes of workspace himuon_grouped_wgrad needs for operands of these shapes
 * (the pointers are not read): at most 16 MiB.  Host-side only. */
himuon_status_t himuon_grouped_wgrad_workspace(const himuon_matrix_t* X, const himuon_matrix_t* D, int32_t n,
                                               himuon_dtype_t dt, size_t* bytes);

/* Element type of a device array of vocabulary ids. */
typedef enum himuon_index {
    HIMUON_I32 = 0,
    HIMUON_I64 = 1
} himuon_index_t;

/*
 * himuon_distill - distillation from a teacher's top logits: the loss of each
 * row and, optionally, its gradient in the same call.
 *
 * With s = Z / temperature and q = softmax(s) over the V columns of a row, and
 * teacher entries (i_j, t_j), j = 1..k, of that row:
 *     p_j  = softmax over the row's entries of t_j / temperature
 *                                                   (normalize != 0), or
 *     p_j  = exp(t_j)                               (normalize == 0; t_j are
 *            log probabilities, taken as they stand)
 *     loss = weight * sum_j p_j (log p_j - log q[i_j])
 *     dZ_v = weight / temperature * (P q_v - sum_{j: i_j = v} p_j),  P = sum_j p_j
 *
 * Z        : N x V student logits.
 * idx      : device array N x k of ids, of type it.  An id outside [0, V)
 *            marks an absent entry.  An id may occur more than once in a row.
 * T        : N x k fp32 teacher values (row stride T->ld).  -inf is p_j = 0.
 * temperature : finite, above 4.3e-39.
 * weight   : device array of N fp32, or NULL (all 1).
 * loss     : device array of N fp32, written.
 * lse      : device array of N x 2 fp32, written, or NULL: log sum exp of s
 *            rounded to fp32, and what that rounding lost (a row masked by the
 *            type's lowest value would lose it all), for himuon_distill_grad.
 *            The row's largest s enters as the fp32 product of the logit and
 *            1 / temperature, held to fp32's finite range.
 * dZ       : N x V in dt, written, or NULL.  It may be Z itself (the same
 *            pointer and ld); any other overlap is refused.
 * workspace: device scratch of at least himuon_distill_workspace bytes,
 *            16-byte aligned; may be NULL when that is 0.
 * A row whose weight is 0, or that has no entry with p_j > 0 (in fp32:
 * exp(t_j) is 0 from about -104 down), counts nothing: its loss, lse and
 * gradient are 0 whatever it holds.  In the other rows a logit
 * of -inf has q = 0 (an entry there gives the loss +inf); NaN or +inf logits
 * make that row's results NaN.  k up to HIMUON_MAX_ENTRIES, V up to 2^29.
 * Errors: HIMUON_ERR_INVALID_ARGUMENT, HIMUON_ERR_UNSUPPORTED (dtype, index
 * type, k above the maximum), HIMUON_ERR_LAYOUT, HIMUON_ERR_OVERLAP,
 * HIMUON_ERR_WORKSPACE, HIMUON_ERR_HIP.
 */
#define HIMUON_MAX_ENTRIES 1024
himuon_status_t himuon_distill(const himuon_matrix_t* Z, const void* idx, himuon_index_t it, const himuon_matrix_t* T,
                               float temperature, int32_t normalize, const float* weight, float* loss, float* lse,
                               const himuon_matrix_t* dZ, himuon_dtype_t dt, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Bytes of workspace himuon_distill needs for logits of this shape (the
 * pointer is not read), with a gradient or without.  Host-side only. */
himuon_status_t himuon_distill_workspace(const himuon_matrix_t* Z, himuon_dtype_t dt, int32_t with_grad,
                                         size_t* bytes);

/*
 * himuon_distill_grad - the gradient alone, from the lse of a himuon_distill
 * call on the same inputs.  g is the device array of N fp32 gradients of the
 * unweighted row losses (dL/dloss_i, times the row's weight if one was used);
 * it takes the place of weight above.  Rows with g = 0 or without entries get
 * zeros.
 */
himuon_status_t himuon_distill_grad(const himuon_matrix_t* Z, const void* idx, himuon_index_t it,
                                    const himuon_matrix_t* T, float temperature, int32_t normalize, const float* lse,
                                    const float* g, const himuon_matrix_t* dZ, himuon_dtype_t dt, void* stream);

/*
 * himuon_token_logprobs - log probabilities of given tokens, with the entropy
 * and the top alternatives of every row.
 *
 * With s = Z / temperature, lse = log sum_v exp(s_v), q = exp(s - lse):
 *     logp    = s[token] - lse
 *     entropy = -sum_v q_v log q_v            (a term with q_v = 0 is 0)
 *     top_idx, top_logp: the ids of the `top` largest logits, largest first
 *              and equal ones by the lowest id, and their log probabilities
 *
 * Z        : N x V logits.
 * tokens   : device array of N ids of type it, or NULL (then logp must be
 *            NULL).  A row whose token lies outside [0, V) is skipped: logp,
 *            entropy and lse are 0, top_idx -1 and top_logp -inf.
 * top      : 0 <= top <= min(V, HIMUON_MAX_TOP).
 * logp, entropy : device arrays of N fp32, written; each may be NULL.
 * lse      : device array of N x 2 fp32, written, or NULL (as for himuon_distill).
 * top_idx, top_logp  : device arrays N x top of int32 and fp32, written; may
 *            be NULL when top is 0.
 * workspace: at least himuon_token_logprobs_workspace bytes, 16-byte aligned;
 *            may be NULL when that is 0.
 * A logit of -inf has q = 0 and log probability -inf (so does every id of a
 * row that holds nothing else; its lse is -inf and its entropy 0).  A NaN or
 * +inf makes the row's values NaN; NaN ranks with -inf among the alternatives.
 * Errors as for himuon_distill.
 */
#define HIMUON_MAX_TOP 64
himuon_status_t himuon_token_logprobs(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it,
                                      float temperature, int32_t top, float* logp, float* entropy, float* lse,
                                      int32_t* top_idx, float* top_logp, himuon_dtype_t dt, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Bytes of workspace himuon_token_logprobs needs for logits of this shape (the
 * pointer is not read).  Host-side only. */
himuon_status_t himuon_token_logprobs_workspace(const himuon_matrix_t* Z, int32_t top, himuon_dtype_t dt,
                                                size_t* bytes);

/*
 * himuon_token_logprobs_grad - the gradient of the logits through logp and
 * entropy:
 *     dZ_v = (g_logp ([v = token] - q_v) - g_entropy q_v (log q_v + entropy)) / temperature
 *
 * lse, entropy : device arrays of N x 2 and N fp32 from himuon_token_logprobs
 *            on the same inputs (entropy may be NULL when g_entropy is).
 * g_logp, g_entropy : device arrays of N fp32, either may be NULL (zero).
 *            tokens may be NULL when g_logp is.
 * dZ       : N x V in dt, written; may be Z itself.
 * A skipped row, and one whose two gradients are 0, gets zeros.
 */
himuon_status_t himuon_token_logprobs_grad(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it,
                                           float temperature, const float* lse, const float* entropy,
                                           const float* g_logp, const float* g_entropy, const himuon_matrix_t* dZ,
                                           himuon_dtype_t dt, void* stream);

/* Static description of a status code (never NULL). */
const char* himuon_status_string(himuon_status_t s);

/* hipError_t of the most recent HIMUON_ERR_HIP on this thread (0 if none). */
int32_t himuon_last_hip_error(void);

/* Library version as major * 10000 + minor * 100 + patch. */
int32_t himuon_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HIMUON_H */
