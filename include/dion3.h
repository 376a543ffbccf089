/*
 * dion3.h -- C ABI of libdion3.so, the Dion3 optimizer step on AMD gfx950.
 *
 * The step (source: "Dion3: Full-Stack Orthogonal Updates", agihunt.info
 * summary, level-1 and level-3 paragraphs; the paper abstract on
 * arxivlens.com / scholarbro.com):
 *   1. score every row of the momentum matrix M (n x m) by its l1 norm;
 *   2. select the k = ceil(f n) best rows (ties: lowest row index);
 *   3. orthogonalize the selected k x m submatrix X with Gram Newton-Schulz:
 *      the quintic iteration runs on the small symmetric Gram R = X X^T
 *      (X^T X when k > m), restarting once (iteration 3 by default) from
 *      X <- Q X, R <- X X^T, Q <- I, and only then is Q multiplied back
 *      onto X; fp16 storage, fp32 accumulation;
 *   4. W[S] <- W[S] - lr * O for the selected rows only, and
 *      M[S] <- mu * M[S] (one fp32 multiply) for the selected rows only.
 *
 * Conventions for every entry point:
 *   - Matrices are row-major.  "Rows" are dim 0 (output neurons).
 *   - Every data pointer is a DEVICE pointer owned by the caller.  The
 *     library never allocates or frees device memory: scratch lives in the
 *     caller's workspace `ws` (at least dion3_workspace_size() bytes,
 *     256-byte aligned).
 *   - fp16 data is IEEE binary16 passed as uint16_t.
 *   - `stream` is a hipStream_t (NULL: the null stream).  Calls only enqueue
 *     work on `stream` and return without synchronizing.
 *   - Errors are status codes; nothing aborts or throws across the ABI.  All
 *     argument checks run before the first launch, so on any error W, M and
 *     the outputs are untouched.
 *   - NaN or Inf in M or X gives undefined results (no check is made).
 *   - Concurrent calls are safe when their workspaces and outputs are
 *     disjoint.  The library's only mutable global state is the thread-local
 *     last HIP error and the optional timing trace (dion3_trace_*).
 *   - Within one call the matrices written (W, M and, for the normalized
 *     step, V; every matrix of a megabatch) must not overlap each other in
 *     memory; W and M must not alias.  Inputs that are only read (G, and X
 *     of dion3_gram_ns) may alias outputs: they are consumed first.
 */
#ifndef DION3_H
#define DION3_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DION3_API __attribute__((visibility("default")))
#else
#define DION3_API
#endif

typedef enum {
  DION3_OK = 0,
  DION3_ERR_ARG = -1,          /* a null required pointer or an out-of-range size/parameter:
                                  any size below 1, k outside [1, n], ld < m, a schedule outside
                                  its stated ranges.  Sizes are checked in that order, so k = 0
                                  or k > n is an argument error even where n or m also exceeds
                                  DION3_MAX_DIM */
  DION3_ERR_WORKSPACE = -2,    /* ws is NULL, misaligned or smaller than dion3_workspace_size() */
  DION3_ERR_UNSUPPORTED = -3,  /* a shape beyond the library's limits (sizes that are
                                  otherwise valid): a dimension above DION3_MAX_DIM, or a
                                  zero-padded per-matrix block (the selected rows, padded to
                                  multiples of 128, or the Gram side) of 2^31 bytes or more, or
                                  a product whose 128 x 128 output tiles over the whole batch
                                  exceed 2^31 - 1; with DION3_PATH_FUSED, also a Gram side
                                  min(k, m) above 128 */
  DION3_ERR_HIP = -4           /* a HIP call or launch failed; see dion3_last_hip_error() */
} dion3_status;

#define DION3_MAX_ITERS 16
#define DION3_MAX_RESTARTS 4
#define DION3_MAX_DIM (1 << 20)   /* n, m, k each at most this */
#define DION3_MAX_BATCH 65535
#define DION3_MAX_GROUPS 64       /* shape groups in one dion3_step_groups call */

/* Newton-Schulz schedule.  Iteration t (1-based) uses the quintic
 * coefficients abc[t-1] = (a, b, c): Z = a I + b R + c R^2.  An iteration
 * listed in restart_at[0..n_restart-1] first materializes X <- Q X,
 * recomputes R <- X X^T and resets Q <- I ("Dion3: Full-Stack Orthogonal
 * Updates", agihunt.info, level-1 paragraph: one restart at the 3rd
 * iteration).  Valid: 1 <= iters <= 16, 0 <= n_restart <= 4, each restart
 * index in [2, iters], strictly increasing.  eps >= 0 is added to ||X||_F in
 * the normalization X / (||X||_F + eps). */
typedef struct {
  int32_t iters;
  int32_t n_restart;
  int32_t restart_at[DION3_MAX_RESTARTS];
  float abc[DION3_MAX_ITERS][3];
  float eps;
  int32_t method;   /* DION3_NS_GRAM (default) or DION3_NS_STANDARD */
  int32_t path;     /* DION3_PATH_AUTO (default), _TILED or _FUSED */
} dion3_ns_cfg;

/* method: DION3_NS_GRAM iterates on the Gram matrix (the level-1 paragraph);
 * DION3_NS_STANDARD runs the standard quintic iteration on X itself,
 * X <- a X + (b A + c A^2) X with A = X X^T, on the same fp16 MFMA kernels
 * (the Muon baseline the pages compare against; restarts do not apply). */
#define DION3_NS_GRAM 0
#define DION3_NS_STANDARD 1

/* path (Gram method only): how the Gram iteration is launched.
 * DION3_PATH_TILED: one tiled MFMA product per step of the iteration (about
 *   20 launches per call, every grid spread over the whole GPU).
 * DION3_PATH_FUSED: one launch, one workgroup per matrix running the whole
 *   iteration with R, Z, Q in LDS (for Gram sides up to 64 one wave runs
 *   every s x s product); only when the Gram side min(k, m) is at most 128,
 *   else DION3_ERR_UNSUPPORTED.  Its result is bitwise identical to the
 *   tiled path (same products, same accumulation order, same roundings).
 * DION3_PATH_AUTO: the fused path where it is allowed and expected to be
 *   faster (Gram side <= 128 and enough matrices or short enough rows for
 *   one workgroup each), the tiled path otherwise.
 * The standard method always runs tiled. */
#define DION3_PATH_AUTO 0
#define DION3_PATH_TILED 1
#define DION3_PATH_FUSED 2

/* Default schedule: Gram Newton-Schulz, 5 iterations of Muon's quintic
 * (3.4445, -4.7750, 2.0315), one restart at iteration 3, eps = 1e-7. */
DION3_API void dion3_ns_cfg_default(dion3_ns_cfg* cfg);

/* sizeof(dion3_ns_cfg) as this library was built, so that a binding can
 * check its own copy of the struct before passing one. */
DION3_API size_t dion3_ns_cfg_size(void);

/* k = ceil(f * n) (level-3 paragraph of the agihunt summary), computed in
 * exact rationals: f is read as the nearest fraction with denominator
 * <= 2^20 (so 0.07 * 100 gives 7, not 8).  The result is clamped to [1, n].
 * Returns -1 if n < 1 or f is not finite and positive. */
DION3_API int64_t dion3_k_from_fraction(double f, int64_t n);

/* Workspace bytes needed by dion3_row_select, dion3_gram_ns, dion3_step
 * and dion3_step_megabatch for `batch` matrices of n x m with k selected
 * rows (for dion3_gram_ns pass n = k).  Host-only; no device work. */
DION3_API dion3_status dion3_workspace_size(int32_t batch, int64_t n, int64_t m, int64_t k, size_t* bytes);

/* Steps 1-2 on `batch` matrices stored back to back: M[b] starts at
 * M + b * n * ld (fp32, row stride ld >= m).  Writes idx[b * k + j]
 * (int32, the k selected rows of matrix b in ascending order) and, when
 * scores is not NULL, scores[b * n + i] = sum_j |M[b][i][j]| (fp64). */
DION3_API dion3_status dion3_row_select(const float* M, int32_t batch, int64_t n, int64_t m, int64_t ld,
                              int64_t k, int32_t* idx, double* scores,
                              void* ws, size_t ws_bytes, void* stream);

/* Step 3 alone on `batch` fp16 matrices X[b] (k x m, contiguous, X + b*k*m):
 * normalizes each by its Frobenius norm, runs Gram Newton-Schulz with `cfg`
 * (NULL: the default) and writes O[b] (k x m fp16, contiguous). */
DION3_API dion3_status dion3_gram_ns(const uint16_t* X, uint16_t* O, int32_t batch, int64_t k, int64_t m,
                           const dion3_ns_cfg* cfg, void* ws, size_t ws_bytes, void* stream);

/* The whole step on one matrix: W and M are fp32 n x m with row stride ld.
 * lr is the final step size (the caller applies the 1/sqrt(f) scaling of
 * the level-3 paragraph); mu is the momentum decay of the selected rows.
 * Rows outside the selected set are never written.  Optional outputs (may
 * be NULL): idx_out[k] (int32 ascending) and O_out (k x m fp16, the
 * orthogonalized update before scaling by lr). */
DION3_API dion3_status dion3_step(float* W, float* M, int64_t n, int64_t m, int64_t ld, int64_t k,
                        float lr, float mu, const dion3_ns_cfg* cfg,
                        int32_t* idx_out, uint16_t* O_out,
                        void* ws, size_t ws_bytes, void* stream);

/* The whole step on `batch` same-shape matrices in one call ("megabatching",
 * level-4 paragraph of the agihunt summary, reduced to one GPU: one launch
 * sequence per shape group).  W and M are DEVICE arrays of `batch` device
 * pointers.  Optional outputs: idx_out[batch][k], O_out[batch][k][m].
 * Results equal `batch` separate dion3_step calls bit for bit. */
DION3_API dion3_status dion3_step_megabatch(float* const* W, float* const* M, int32_t batch,
                                  int64_t n, int64_t m, int64_t ld, int64_t k,
                                  float lr, float mu, const dion3_ns_cfg* cfg,
                                  int32_t* idx_out, uint16_t* O_out,
                                  void* ws, size_t ws_bytes, void* stream);

/* The step with the gradient accumulated into the momentum buffer first:
 * M <- M + G (one fp32 add per element, every row of M), then the step as in
 * dion3_step / dion3_step_megabatch on the updated M.  Error feedback keeps
 * the unselected rows of the buffer for later steps and decays only the
 * selected ones ("Dion3: Full-Stack Orthogonal Updates", agihunt.info,
 * level-3 paragraph), so the buffer is a running sum of gradients.  The
 * addition is fused into the row scoring, which reads M and G once.  G has
 * the shape and row stride of M and is not written; for the megabatch form
 * it is a DEVICE array of `batch` device pointers.  Results equal adding G
 * to M in fp32 and then calling dion3_step, bit for bit. */
DION3_API dion3_status dion3_step_accum(float* W, float* M, const float* G, int64_t n, int64_t m,
                                        int64_t ld, int64_t k, float lr, float mu,
                                        const dion3_ns_cfg* cfg, int32_t* idx_out,
                                        uint16_t* O_out, void* ws, size_t ws_bytes, void* stream);
DION3_API dion3_status dion3_step_megabatch_accum(float* const* W, float* const* M,
                                                  const float* const* G, int32_t batch, int64_t n,
                                                  int64_t m, int64_t ld, int64_t k, float lr,
                                                  float mu, const dion3_ns_cfg* cfg,
                                                  int32_t* idx_out, uint16_t* O_out, void* ws,
                                                  size_t ws_bytes, void* stream);

/* Per-neuron normalization of the update.  The pages say that Dion3
 * inherits NorMuon's per-neuron normalization ("Dion3 Cuts Muon Optimizer
 * Time by Up to 6x", quasa.io, section "Dion3's fastest path is a combined
 * systems stack") and that it runs in float32 ("Dion3: Full-Stack
 * Orthogonal Updates", agihunt.info, limitations paragraph), without a
 * formula.  Reading implemented: for the selected rows S and orthogonalized
 * rows O (k x m) of one matrix with a float32 state V (n entries, one per
 * row, caller-owned, zero before the first step):
 *   q_i = mean_j O_ij^2;  V[S_i] <- beta2 V[S_i] + (1 - beta2) q_i;
 *   U_i = O_i / (sqrt(V[S_i]) + eps)  (0 for a zero row with zero state);
 *   U <- U ||O||_F / ||U||_F  (the step keeps O's norm);
 *   W[S] <- W[S] - lr U.  Rows of V outside S are not written. */
typedef struct {
  float beta2;   /* 0 <= beta2 < 1 */
  float eps;     /* >= 0, added to sqrt(V) */
} dion3_norm_cfg;

/* The megabatch step with per-neuron normalization.  W, M, V are DEVICE
 * arrays of `batch` device pointers (V[b]: n floats); G is NULL or such an
 * array of gradients accumulated first as in dion3_step_megabatch_accum.
 * O_out, when not NULL, receives O before the normalization.  The workspace
 * is the one dion3_workspace_size gives for the same shapes.
 * DION3_ERR_ARG also for a NULL V or norm, beta2 outside [0, 1) or eps < 0. */
DION3_API dion3_status dion3_step_megabatch_norm(float* const* W, float* const* M,
                                                 const float* const* G, float* const* V,
                                                 int32_t batch, int64_t n, int64_t m, int64_t ld,
                                                 int64_t k, float lr, float mu,
                                                 const dion3_ns_cfg* cfg,
                                                 const dion3_norm_cfg* norm, int32_t* idx_out,
                                                 uint16_t* O_out, void* ws, size_t ws_bytes,
                                                 void* stream);

/* One shape group of a whole-model step (dion3_step_groups): `batch`
 * matrices of n x m (row stride ld) with k selected rows each and step size
 * lr.  W, M (and G, V when used) are DEVICE arrays of `batch` device
 * pointers, as in dion3_step_megabatch_accum / _norm.  G: NULL, or the
 * gradients accumulated first (M <- M + G).  V: the per-neuron
 * normalization states (n floats per matrix); required when the call is
 * given a dion3_norm_cfg, ignored otherwise.  idx_out ([batch][k] int32) and
 * O_out ([batch][k][m] fp16) are optional outputs as in the megabatch call. */
typedef struct {
  float* const* W;
  float* const* M;
  const float* const* G;
  float* const* V;
  int64_t n, m, ld, k;
  int32_t batch;
  float lr;
  int32_t* idx_out;
  uint16_t* O_out;
} dion3_group;

/* sizeof(dion3_group) as this library was built (for bindings). */
DION3_API size_t dion3_group_size(void);

/* Workspace bytes for dion3_step_groups over these groups and this schedule
 * (cfg NULL: the default).  Only the sizes of each group are read.  The
 * status codes are those of dion3_step_groups' shape checks. */
DION3_API dion3_status dion3_workspace_size_groups(const dion3_group* groups, int32_t ngroups,
                                                   const dion3_ns_cfg* cfg, size_t* bytes);

/* The step over a whole model's shape groups in one call (the host array
 * `groups`, 1 <= ngroups <= DION3_MAX_GROUPS).  Megabatching ("Dion3:
 * Full-Stack Orthogonal Updates", agihunt.info, level-4 paragraph) carried
 * one level further on one GPU: groups whose Gram sides are equal (s =
 * min(k, m); e.g. the attention and down-projection matrices of a
 * transformer at one fraction) may share one set of s x s matrices, where a
 * launch-round cost model says that their products (the polynomial and the
 * symmetric products of the level-2 paragraph) run no slower as one; the
 * side sets then run the iteration in step, each s x s product one launch
 * over every set and each Gram one launch over every group (the
 * multiply-backs, which write each group's own rows, run per group).  With
 * the 128-matrix batch of attention-shaped matrices and the 32 of
 * down-projection shape of a 7B-like model at f = 1/4 that is 8 symmetric,
 * 5 polynomial and 2 Gram launches per step instead of 18, 10 and 6 (the
 * two independent products that read the same polynomial also share one).
 * norm: NULL, or the
 * per-neuron normalization of dion3_step_megabatch_norm for every group.
 * Results equal calling dion3_step_megabatch (_accum, _norm) once per group
 * with the same arguments, bit for bit.  Matrices written by different
 * groups must not overlap.  All checks (every group, then the workspace)
 * run before the first launch. */
DION3_API dion3_status dion3_step_groups(const dion3_group* groups, int32_t ngroups, float mu,
                                         const dion3_ns_cfg* cfg, const dion3_norm_cfg* norm,
                                         void* ws, size_t ws_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the
 * megabatched step of dion3_step_megabatch with the same arguments and
 * results bit for bit, but no workspace argument.  Its scratch is a static
 * device array of DION3_STATIC_SCRATCH_BYTES in the library, one per GPU
 * (held until the process ends); the call allocates nothing.  Every call on
 * one GPU shares that GPU's array, so calls that overlap on one GPU (other
 * streams, other threads) race; serialize them.  Nothing in the array needs
 * to start at zero: every region the step reads is written first in the same
 * call.  The stream must belong to the current device.
 * DION3_ERR_WORKSPACE: the call needs more than DION3_STATIC_SCRATCH_BYTES
 * (dion3_workspace_size for the same shapes), checked before any launch.
 * DION3_ERR_ARG also when the stream belongs to another device; the other
 * status codes are dion3_step_megabatch's. */
#define DION3_STATIC_SCRATCH_BYTES (64u << 20)
DION3_API dion3_status dion3_step_megabatch_noalloc(float* const* W, float* const* M, int32_t batch,
                                                    int64_t n, int64_t m, int64_t ld, int64_t k,
                                                    float lr, float mu, const dion3_ns_cfg* cfg,
                                                    int32_t* idx_out, uint16_t* O_out,
                                                    void* stream);

/* The symmetric products of the level-2 paragraph, usable on their own.
 *
 * dion3_syrk_f16: R[b] = A[b] A[b]^T for `batch` fp16 matrices A[b]
 * (rows x cols, row stride lda, batch stride rows*lda).  R[b] is rows x rows
 * fp16 with row stride ldr (batch stride rows*ldr); only lower-triangle
 * tiles are computed and each is mirrored, so R is exactly symmetric.
 * rows and cols must be multiples of 128 and lda, ldr multiples of 8. */
DION3_API dion3_status dion3_syrk_f16(const uint16_t* A, uint16_t* R, int32_t batch, int64_t rows,
                            int64_t cols, int64_t lda, int64_t ldr, void* stream);

/* dion3_symm_f16 ("A^2 + B"): C[b] = alpha A[b] B[b] + beta D[b] + gamma I
 * for symmetric, commuting s x s fp16 matrices A[b], B[b] (so the product is
 * symmetric) and a symmetric D[b]; D may be NULL when beta == 0.  All four share row stride ld and
 * batch stride s*ld; s must be a multiple of 128, ld a multiple of 8.  Only
 * lower-triangle tiles are computed, then mirrored.  C must not alias A, B
 * or D. */
DION3_API dion3_status dion3_symm_f16(const uint16_t* A, const uint16_t* B, const uint16_t* D, uint16_t* C,
                            int32_t batch, int64_t s, int64_t ld, float alpha, float beta,
                            float gamma, void* stream);

/* ---------------------------------------------------------------------------
 * Operators of the layers whose weights the step updates: the norm before a
 * linear layer, the layer's product with its epilogue, both gradients, and
 * activations held in 8 bits between the forward and the backward pass.  The
 * weight gradient is summed in fp32 and may be added straight into the
 * momentum buffer M, which the step then takes as it is (dion3_step: no G).
 *
 * T tokens; matrices are row-major with a row stride (ld) of their own.
 * 16-bit data (`dtype`: DION3_BF16 or DION3_F16) is passed as void*; every
 * pointer is aligned to its element size (8-bit data: 16 bytes).  Any side
 * from 1 and any row stride that holds the row is taken; rows that are
 * 16-byte aligned with sides that are multiples of 8 are fastest (over others
 * the products take a fifth to three fifths longer, or copy them into the
 * workspace first, whichever is expected to take less).  T = 0 is
 * valid: nothing is written, except that gradients over no tokens are zero.
 * Statistics, products and column sums are held in fp32 and added in an order
 * fixed by the sizes, strides and alignment alone; every output is rounded
 * once.  Outputs must not overlap inputs or each other except where said.
 * NaN and infinities propagate as in the formulas.
 * DION3_ERR_ARG: a null required pointer, a negative T, a side below 1, a
 * row stride below the row, an unknown type or activation, an unaligned
 * pointer.  DION3_ERR_UNSUPPORTED: T above DION3_MAX_TOKENS, a side above
 * DION3_MAX_DIM, a row stride above 2^21 or a matrix of more than 2^38 elements.
 * DION3_ERR_WORKSPACE: as elsewhere; a call whose workspace size is 0 takes
 * ws = NULL. */
#define DION3_F32 0
#define DION3_BF16 1
#define DION3_F16 2

#define DION3_ACT_NONE 0
#define DION3_ACT_RELU 1
#define DION3_ACT_GELU 2        /* z (1 + erf(z / sqrt 2)) / 2 */
#define DION3_ACT_GELU_TANH 3   /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
#define DION3_ACT_SILU 4        /* z / (1 + exp(-z)) */

#define DION3_MAX_TOKENS (1 << 24)

/* The 8-bit format.  Columns are padded with zeros to mp = m rounded up to
 * DION3_F8_BLOCK; Q holds T x mp bytes of e4m3 (contiguous), S one scale byte
 * per block of DION3_F8_BLOCK columns (T x mp / DION3_F8_BLOCK, contiguous).
 * A value is q * 2^(s - 127).  The scale is the smallest power of two
 * that brings the block's largest finite magnitude to 448 or below (at least
 * 2^-127), so that nothing saturates, and q is rounded to nearest even.
 * Infinities and NaN become NaN and leave the scale alone.  In a block whose
 * scale is the type's last (2^120; 2^8 for fp16) magnitudes end at 240
 * scales, so that every value fits its type again. */
#define DION3_F8_BLOCK 32

/* h = X + R, rstd = 1 / sqrt(mean_j h_j^2 + eps), Y = h * rstd * w per row.
 * H receives h rounded to dtype, and the statistics and Y are those of the
 * rounded h.  R and H are both given, or both NULL (then h = X); H may be X
 * or R.  w has m entries of wtype (DION3_F32 or dtype).  Outputs: Y and / or
 * Q and S (the packed form of Y's rounded values), and rstd (T floats)
 * unless NULL.  The squares are summed in fp32 as they are: a row whose sum
 * passes its largest value (one of |h| = 1.9e19 does) gets rstd = 0, and h
 * below 1e-23 count as zeros. */
DION3_API dion3_status dion3_add_rms_norm(const void* X, int64_t ldx, const void* R, int64_t ldr,
                                          const void* w, int32_t wtype, void* H, int64_t ldh,
                                          void* Y, int64_t ldy, uint8_t* Q, uint8_t* S, float* rstd,
                                          int64_t T, int64_t m, float eps, int32_t dtype,
                                          void* stream);

/* Its gradient, from h and rstd as the forward pass left them.  With a = w dY
 * and u = h rstd: dX = rstd (a - u mean_j(a_j u_j)) + dH, the gradient of both
 * X and R (dH: the gradient that reaches h past the norm, or NULL), and
 * dw = sum over tokens of dY u.  dX and dw may each be NULL, not both; dX may
 * be dY or dH. */
DION3_API dion3_status dion3_add_rms_norm_grad_workspace_size(int64_t T, int64_t m, size_t* bytes);
DION3_API dion3_status dion3_add_rms_norm_grad(const void* dY, int64_t lddy, const void* H,
                                               int64_t ldh, const float* rstd, const void* w,
                                               int32_t wtype, const void* dH, int64_t lddh, void* dX,
                                               int64_t lddx, float* dw, int64_t T, int64_t m,
                                               int32_t dtype, void* ws, size_t ws_bytes,
                                               void* stream);

/* X (dtype, or DION3_F32) into the 8-bit format, and its values back. */
DION3_API dion3_status dion3_pack_f8(const void* X, int64_t ldx, uint8_t* Q, uint8_t* S, int64_t T,
                                     int64_t m, int32_t dtype, void* stream);
DION3_API dion3_status dion3_unpack_f8(const uint8_t* Q, const uint8_t* S, void* Y, int64_t ldy,
                                       int64_t T, int64_t m, int32_t dtype, void* stream);

/* z = X W^T + bias, Y = act(z) + R, with X: T x m, W: n x m, Y: T x n.  bias
 * (n entries of bias_type, DION3_F32 or dtype), R (T x n) and Z may be NULL;
 * Z receives z rounded to dtype (act reads it unrounded).  Y may be R.  The
 * workspace depends on the pointers' alignment only, not on their contents. */
DION3_API dion3_status dion3_linear_workspace_size(const void* X, int64_t ldx, const void* W,
                                                   int64_t ldw, int64_t T, int64_t n, int64_t m,
                                                   size_t* bytes);
DION3_API dion3_status dion3_linear(const void* X, int64_t ldx, const void* W, int64_t ldw,
                                    const void* bias, int32_t bias_type, const void* R, int64_t ldr,
                                    void* Y, int64_t ldy, void* Z, int64_t ldz, int64_t T, int64_t n,
                                    int64_t m, int32_t act, int32_t dtype, void* ws, size_t ws_bytes,
                                    void* stream);

/* dZ = dY act'(z) and db = sum over tokens of dY act'(z) (fp32, n entries,
 * summed before dZ's rounding).  z comes from Z, or from its 8-bit form ZQ,
 * ZS (whose values stand for z, zeros too: a z below 4.4e-6 of its block's
 * largest may be one, where the slope of relu is 0); neither is read for
 * DION3_ACT_NONE.  dZ and db may each be NULL, not both; dZ may be dY or Z.
 * The workspace is used for db only. */
DION3_API dion3_status dion3_act_grad_workspace_size(int64_t T, int64_t n, size_t* bytes);
DION3_API dion3_status dion3_act_grad(const void* dY, int64_t lddy, const void* Z, int64_t ldz,
                                      const uint8_t* ZQ, const uint8_t* ZS, void* dZ, int64_t lddz,
                                      float* db, int64_t T, int64_t n, int32_t act, int32_t dtype,
                                      void* ws, size_t ws_bytes, void* stream);

/* dX = dZ W (+ R, T x m, or NULL), with dZ: T x n, W: n x m.  dX may be R. */
DION3_API dion3_status dion3_linear_grad_input_workspace_size(const void* dZ, int64_t lddz,
                                                              const void* W, int64_t ldw, int64_t T,
                                                              int64_t n, int64_t m, size_t* bytes);
DION3_API dion3_status dion3_linear_grad_input(const void* dZ, int64_t lddz, const void* W,
                                               int64_t ldw, const void* R, int64_t ldr, void* dX,
                                               int64_t lddx, int64_t T, int64_t n, int64_t m,
                                               int32_t dtype, void* ws, size_t ws_bytes,
                                               void* stream);

/* G = dZ^T X, or with accumulate != 0 G <- G + dZ^T X, in fp32: dZ: T x n,
 * G: n x m.  X is T x m of dtype when S is NULL; otherwise X and S are an
 * 8-bit checkpoint (ldx is not read), whose values enter the product rounded
 * to dtype (exact unless they leave its range).  G may be the momentum M of
 * dion3_step. */
DION3_API dion3_status dion3_linear_grad_weight_workspace_size(const void* dZ, int64_t lddz,
                                                               const void* X, int64_t ldx,
                                                               const uint8_t* S, int64_t T,
                                                               int64_t n, int64_t m, size_t* bytes);
DION3_API dion3_status dion3_linear_grad_weight(const void* dZ, int64_t lddz, const void* X,
                                                int64_t ldx, const uint8_t* S, float* G, int64_t ldg,
                                                int32_t accumulate, int64_t T, int64_t n, int64_t m,
                                                int32_t dtype, void* ws, size_t ws_bytes,
                                                void* stream);

/* ---------------------------------------------------------------------------
 * Embedding lookup with scaling, and its gradient.
 *
 * token: T integers of token_bits (32 or 64) bits; W: n x m of wtype, Y: T x m
 * of dtype (each DION3_F32, _BF16 or _F16; wtype is DION3_F32 or dtype).
 *   Y[t] = scale W[token[t]], rounded once.
 * A token outside [0, n) stands for none (padding, or a row of another part of
 * the vocabulary): its row of Y is zeros, and it sends no gradient.
 *
 * The gradient: dW[v] = scale times the sum of dY[t] over the t with token[t]
 * = v (fp32, n x m; zeros for a row without tokens), or with accumulate != 0
 * that is added to dW, and rows without tokens are neither read nor written.
 * Sums are held in fp32, those of a token with more than 64 rows in parts that
 * are added up in 64 bits, without atomics, in an order fixed by the tokens.
 * Errors: as for the layers' operators, but row strides up to 2^38; scale must
 * be finite. */
DION3_API dion3_status dion3_embedding(const void* token, int32_t token_bits, const void* W,
                                       int64_t ldw, int32_t wtype, void* Y, int64_t ldy, int64_t T,
                                       int64_t n, int64_t m, float scale, int32_t dtype,
                                       void* stream);
DION3_API dion3_status dion3_embedding_grad_workspace_size(int64_t T, int64_t n, int64_t m,
                                                           size_t* bytes);
DION3_API dion3_status dion3_embedding_grad(const void* token, int32_t token_bits, const void* dY,
                                            int64_t lddy, float* dW, int64_t ldw,
                                            int32_t accumulate, int64_t T, int64_t n, int64_t m,
                                            float scale, int32_t dtype, void* ws, size_t ws_bytes,
                                            void* stream);

/* ---------------------------------------------------------------------------
 * Norms of queries and keys per head with the rotation by their positions in
 * the same pass, and the gradient.
 *
 * A side (the queries, or the keys) is T tokens of `heads` heads of D columns:
 * element (t, h, j) of X is X[t ldx + h hsx + j], so that the parts of one
 * product's output, or heads before tokens, are read as they lie; Y and dY
 * likewise.  All are of dtype; w (D entries) is DION3_F32 or of dtype.
 *   rstd = 1 / sqrt(mean_j x_j^2 + eps) and u = x rstd w per head;
 *   the first r columns are turned: (y_a, y_b) = (u_a c - u_b s, u_b c + u_a s)
 *   with c, s the cosine and sine of pos[t] freqs[i] for the pairs i < r / 2,
 *   (a, b) = (i, i + r / 2), or (2 i, 2 i + 1) when interleaved;
 *   the other columns are u.
 * freqs: r / 2 doubles (radians a position); pos: T integers of pos_bits (32
 * or 64) bits.  Angles are computed in 64 bits, statistics in 32, Y is rounded
 * once.  k may be NULL.  Y may be X.
 *
 * The gradient, from X as the forward pass read it: Y receives dX (may be X or
 * dY; NULL: not wanted), dw (2 D floats: those of q's w, then of k's, or NULL)
 * the sums over tokens and heads, in an order fixed by the sizes; k NULL: the
 * second half is zeros.  The workspace is used for dw only.
 * DION3_ERR_ARG, _UNSUPPORTED: as for the layers' operators; r odd, negative
 * or above D; heads below 1; a stride below D where there is more than one;
 * unsupported: D above 1024 (a head takes at most 64 pieces of 16 columns,
 * counted for the turned columns and the others apart), more than 65536
 * heads, a stride above 2^38. */
typedef struct {
  const void* X; int64_t ldx, hsx;
  const void* w;
  const void* dY; int64_t lddy, hsdy;   /* gradient only */
  void* Y; int64_t ldy, hsy;
  int32_t heads;
} dion3_heads;

/* sizeof(dion3_heads) as this library was built (for bindings). */
DION3_API size_t dion3_heads_size(void);

DION3_API dion3_status dion3_qk_norm_rope(const dion3_heads* q, const dion3_heads* k,
                                          const double* freqs, const void* pos, int32_t pos_bits,
                                          int64_t T, int32_t D, int32_t r, int32_t interleaved,
                                          float eps, int32_t wtype, int32_t dtype, void* stream);
DION3_API dion3_status dion3_qk_norm_rope_grad_workspace_size(int64_t T, int32_t hq, int32_t hk,
                                                              int32_t D, int32_t r,
                                                              int32_t interleaved, size_t* bytes);
DION3_API dion3_status dion3_qk_norm_rope_grad(const dion3_heads* q, const dion3_heads* k,
                                               const double* freqs, const void* pos,
                                               int32_t pos_bits, float* dw, int64_t T, int32_t D,
                                               int32_t r, int32_t interleaved, float eps,
                                               int32_t wtype, int32_t dtype, void* ws,
                                               size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens, the entropy and the best alternatives,
 * and the gradient.
 *
 * X holds T rows of n logits of dtype (DION3_F32, _BF16 or _F16) with row
 * stride ldx; z = scale X, held at -FLT_MAX where a finite logit's product
 * passes it (and rounded to fp32 in rows whose maximum is 2^30 or more in
 * magnitude).  target: T integers of target_bits (32 or 64) bits, or NULL; one
 * outside [0, n) marks a row without a token (its logp is 0 and it sends no
 * gradient).
 *   stats[t] = (m, l): m = max_j z_j, l = ln sum_j exp(z_j - m);
 *   logp[t] = (z_target - m) - l (given and NULL together with target);
 *   entropy[t] = -sum_j p_j ln p_j with p_j = exp((z_j - m) - l) (or NULL);
 *   top_logp[t][i], top_index[t][i], i < top <= DION3_MAX_TOP (and n): the
 *   largest logits in order, equal ones by their index, NaN before all.
 * A row whose logits are all -infinity has stats (-infinity, 0), logp and
 * top_logp -infinity, entropy and gradient 0; one with NaN or +infinity (also
 * as the product with scale) has NaN.  The maximum is held apart from the sum
 * so that rows at the type's lowest value keep their probabilities.
 *
 * The gradient: dX_j = scale (g (1[j = target] - p_j) - gH p_j (ln p_j + H))
 * rounded to dtype, with g = dlogp[t] (given and NULL together with target),
 * gH = dentropy[t] (or NULL) and H = entropy[t] (read with dentropy only).
 * dX may be X.
 * Sums are held in fp32 in an order fixed by n.  Errors: as for the layers'
 * operators (sides: n), but row strides up to 2^38 (the last tokens' rows of
 * long sequences, say); top negative or above n is an argument error, above
 * DION3_MAX_TOP unsupported. */
#define DION3_MAX_TOP 64
DION3_API dion3_status dion3_log_probs_workspace_size(int64_t T, int64_t n, int32_t top,
                                                      size_t* bytes);
DION3_API dion3_status dion3_log_probs(const void* X, int64_t ldx, const void* target,
                                       int32_t target_bits, float* logp, float* stats,
                                       float* entropy, float* top_logp, int64_t* top_index,
                                       int64_t T, int64_t n, int32_t top, float scale,
                                       int32_t dtype, void* ws, size_t ws_bytes, void* stream);
DION3_API dion3_status dion3_log_probs_grad(const float* dlogp, const void* X, int64_t ldx,
                                            const void* target, int32_t target_bits,
                                            const float* stats, const float* entropy,
                                            const float* dentropy, void* dX, int64_t lddx,
                                            int64_t T, int64_t n, float scale, int32_t dtype,
                                            void* stream);

/* ---------------------------------------------------------------------------
 * The global norm of many gradients, and their clipping.
 *
 * A gradient is rows x cols elements of dtype (DION3_F32, _BF16 or _F16) with
 * row stride ldg; M, where given, is an fp32 buffer of the same shape with row
 * stride ldm.  (Tensors of any shape without gaps are one row.)  A gradient
 * without elements may have null pointers.  What a call writes must not
 * overlap anything else in the list.
 * DION3_ERR_ARG: a negative count or size, a null or unaligned pointer, a row
 * stride below the row, an unknown type, scale not finite and positive,
 * max_norm negative or NaN.  DION3_ERR_UNSUPPORTED: more than 2^20 gradients
 * or 2^38 elements. */
typedef struct {
  void* G;
  float* M;
  int64_t rows, cols;
  int64_t ldg, ldm;
  int32_t dtype;
} dion3_grad;

/* sizeof(dion3_grad) as this library was built (for bindings). */
DION3_API size_t dion3_grad_size(void);

/* norm = scale sqrt(sum over all gradients of g^2) (one float, rounded once)
 * and, unless NULL, norms[i] = the same of gradient i alone.  Squares are
 * summed in 64 bits in an order fixed by the sizes: no finite gradient
 * overflows the sum, and none is too small for it.  `grads` is a host array;
 * it is read during the call only.  The workspace serves both calls. */
DION3_API dion3_status dion3_grad_norm_workspace_size(const dion3_grad* grads, int32_t count,
                                                      size_t* bytes);
DION3_API dion3_status dion3_grad_norm(const dion3_grad* grads, int32_t count, float scale,
                                       float* norm, float* norms, void* ws, size_t ws_bytes,
                                       void* stream);

/* With that norm and c = 1 where norm <= max_norm, else max_norm / norm (in 64
 * bits, like the products below, which are rounded to fp32 once): each
 * gradient with an M is summed into it, M <- M + c scale G (G is not written),
 * each other one is scaled in place, G <- c scale G rounded to its type.  An
 * infinite norm gives c = 0, a NaN c = NaN.  norm: one float, or NULL.
 * max_norm may be infinite. */
DION3_API dion3_status dion3_clip_grad_norm(const dion3_grad* grads, int32_t count, float max_norm,
                                            float scale, float* norm, void* ws, size_t ws_bytes,
                                            void* stream);

/* Kernel timing trace, for benchmarks.  dion3_trace_enable(capacity > 0)
 * creates 2 * capacity HIP events (no device memory) and starts recording:
 * each kernel the library then launches is timed by events on the caller's
 * stream and noted with its name and the algorithmic work it does on
 * unpadded sizes (flops for the MFMA products, HBM bytes for the row
 * kernels).  Within one library call a kernel's start is the previous
 * kernel's end event, so one event is recorded per kernel and a kernel's
 * time includes its own dispatch; the first kernel of a call, and the first
 * after an untimed copy, records a start event of its own.  Records past
 * the capacity are dropped.  capacity <= 0 stops and frees the trace.
 * dion3_trace_record(i, ...) waits for record i's end event and returns its
 * kernel name (a static string), elapsed ms, flops and bytes; it returns
 * DION3_ERR_HIP when recording either event failed.  The trace is
 * process-wide; it is meant for one benchmarking thread. */
DION3_API dion3_status dion3_trace_enable(int32_t capacity);
DION3_API int32_t dion3_trace_count(void);
DION3_API void dion3_trace_reset(void);
DION3_API dion3_status dion3_trace_record(int32_t i, const char** name, double* ms, double* flops,
                                          double* bytes);

DION3_API const char* dion3_status_string(dion3_status status);

/* hipError_t of the last DION3_ERR_HIP returned on the calling thread (0 if none). */
DION3_API int dion3_last_hip_error(void);

/* Library version, for the binding's load check. */
DION3_API int dion3_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DION3_H */
