/*
 * tsm_gemm.h -- C ABI of the MI355X (gfx950) blocked GEMM library.
 * (The int8 and 4-bit products, the expert routing and the router have sections of
 * their own below.)
 *
 * The operation is the blocked matrix product C = A.B with 16-bit floating-point
 * operands (f16 or bf16), float32 accumulation and a float32 or f16 result.  It
 * is the computation of the 64x128x128 f16 example on "The PTSS Cliff: A Kernel
 * That Won't Build" (sections "The Arithmetic of 'Fully Unrolled K'" and "The
 * Idea: Stage in SLM, Tile K"): every output cell is sum_k A[i][k] * B[k][j],
 * computed by workgroups that each own an output tile and walk K in bounded
 * slices staged through on-chip shared memory (LDS on gfx950).  The masked
 * K-blocked loop with a float32 accumulator and zero padding outside the matrix
 * is the one of the Intel XPU Triton README, section "Use Tensor Descriptors to
 * load tl.dot arguments and save results".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Sizes, leading dimensions and batch strides are counted in ELEMENTS, and
 *    are 64-bit ("A Dumb Triton Runtime Error", Step 1: strides in elements;
 *    Intel XPU Triton README, "Avoid int32 Overflow": offsets are formed in
 *    64 bits).
 *  - A is logically M x K, B is K x N, C is M x N.
 *      row-major A: A[i*lda + k], lda >= K      column-major A: A[k*lda + i], lda >= M
 *      row-major B: B[k*ldb + j], ldb >= N      column-major B: B[j*ldb + k], ldb >= K
 *      C is always row-major:  C[i*ldc + j], ldc >= N
 *  - C is OVERWRITTEN with A.B (no accumulate, no atomics): "A Dumb Triton
 *    Runtime Error", section "Making It Compile, and Why I'd Still Use the
 *    Original", shows read-modify-write into an output that was not zeroed
 *    giving wrong rows.  Elements of C outside the M x N region (the ld padding)
 *    are never written.  K = 0 with M, N > 0 writes zeros (the empty sum).
 *  - Operand elements outside M, N or K never contribute: tiles are loaded
 *    with zero padding ("A Dumb Triton Runtime Error", Step 2, on masking with
 *    the additive identity).
 *  - Pointers are device pointers owned by the caller (e.g. torch tensors).  The
 *    library allocates nothing, keeps no mutable global state and never
 *    synchronises: it enqueues kernels on `stream` (a hipStream_t; NULL = the
 *    null stream) and returns.  Results are valid once the stream reaches them.
 *  - Any 2-byte-aligned operand base and any leading dimension is accepted;
 *    the vector width of the loads is chosen inside the library.  C must be
 *    4-byte aligned for float32 output and 2-byte aligned for f16 output.
 *  - Errors: every argument check runs on the host before any HIP call; on an
 *    error nothing is enqueued and a status code is returned.  No C++ exception
 *    crosses this boundary.  tsm_last_error_detail() names the failed check.
 *
 * Status codes and enums are plain ints so that any FFI can call in.
 */
#ifndef TSM_GEMM_H
#define TSM_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define TSM_SUCCESS 0
#define TSM_ERROR_INVALID_VALUE 1 /* an argument breaks the contract above      */
#define TSM_ERROR_NOT_SUPPORTED 2 /* valid, but beyond this library's limits     */
#define TSM_ERROR_LAUNCH 3        /* the HIP runtime refused or failed a launch */

/* dtype: operand format and output format.  Accumulation is always float32;
 * a 16-bit output is rounded to nearest even from the float32 result. */
#define TSM_F16_F32 0
#define TSM_F16_F16 1
#define TSM_BF16_F32 2
#define TSM_BF16_F16 3
#define TSM_F16_BF16 4
#define TSM_BF16_BF16 5

/* Epilogue activation of gemm_strided_batched_act, applied to the float32
 * result before the output conversion. */
#define TSM_ACT_NONE 0
#define TSM_ACT_RELU 1       /* x > 0 ? x : 0          */
#define TSM_ACT_LEAKY_RELU 2 /* x > 0 ? x : slope * x  */

/* Storage layout of an operand. */
#define TSM_ROW 0
#define TSM_COL 1

/*
 * gemm -- C := A.B for row-major A (M x K) and row-major B (K x N): the product
 * of "The PTSS Cliff", section "The Arithmetic of 'Fully Unrolled K'" (each
 * output cell the sum over k of A[i][k] * B[k][j]), with the K-tiled, LDS-staged
 * blocking of its section "The Idea: Stage in SLM, Tile K".
 *   M, N, K   : sizes, >= 0.
 *   A, lda    : operand A and its leading dimension (>= max(1, K)).
 *   B, ldb    : operand B and its leading dimension (>= max(1, N)).
 *   C, ldc    : result, leading dimension >= max(1, N).
 *   dtype     : operand -> output format: TSM_F16_F32, TSM_F16_F16, TSM_BF16_F32,
 *               TSM_BF16_F16, TSM_F16_BF16 or TSM_BF16_BF16.
 *   stream    : hipStream_t to enqueue on (NULL = null stream).
 * Returns a status code.  M = 0 or N = 0 succeeds without launching.
 * Errors (TSM_ERROR_INVALID_VALUE): negative size; NULL pointer with work to do;
 * leading dimension below the row length; unknown dtype; misaligned pointer;
 * C overlapping A or B.  TSM_ERROR_NOT_SUPPORTED: sizes whose tile grid or
 * element offsets exceed the launch limits (reported, never truncated).
 */
int gemm(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb, void *C,
         int64_t ldc, int dtype, void *stream);

/*
 * gemm_ex -- gemm with an explicit storage layout per operand
 * (layout_a, layout_b in {TSM_ROW, TSM_COL}); gemm is gemm_ex(TSM_ROW, TSM_ROW).
 * The Intel XPU Triton README's matmul signature ("Use Proper Type
 * Annotations") takes a row and a column stride per operand, so either storage
 * order of A and B is the same product; here the two orders that keep one
 * dimension contiguous are offered.
 * A column-major B (element (k, j) at B[j*ldb + k], ldb >= K) makes both operands
 * contiguous along K, the layout the square bf16 product uses.
 */
int gemm_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a, const void *B,
            int64_t ldb, int layout_b, void *C, int64_t ldc, int dtype, void *stream);

/*
 * gemm_strided_batched -- batch independent products, problem z using
 *   A + z*strideA, B + z*strideB, C + z*strideC   (strides in elements, 64-bit).
 * The per-problem slices follow the batched indexing of the Intel XPU Triton
 * README (section "Use Tensor Descriptors to load tl.dot arguments and save
 * results", one expert's slice of a 3-D operand per program); the offsets are
 * formed in 64 bits, as its section "Avoid int32 Overflow" requires once a
 * stride product passes 2^31 (the 8-problem skinny workload's B spans 2^31
 * bytes).
 * strideA or strideB may be 0 (the operand is shared by every problem).
 * strideC must keep the outputs disjoint: strideC >= (M-1)*ldc + N when batch > 1.
 * batch = 0 succeeds without launching.  Other rules as for gemm.
 */
int gemm_strided_batched(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int64_t strideA,
                         const void *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc, int64_t strideC,
                         int64_t batch, int dtype, void *stream);

/* gemm_strided_batched_ex -- gemm_strided_batched with per-operand layouts
 * (as gemm_ex: the README's per-operand strides, restricted to row- or
 * column-major storage).
 * Row bands: one problem (batch 1) of more than one round of 256 x 256 tiles
 * (a round: one tile per CU) whose last round is partly empty may run as two
 * launches on the stream, one after the other: the rows that fill whole rounds
 * on the 256 x 256 kernel, the remaining rows as a problem of their own on the
 * kernel chosen for that problem.  Each element of C is computed by one of the
 * two.  This applies to every plain entry point (gemm to
 * gemm_strided_batched_act, and gemm_strided_batched_ws and _noalloc when they
 * do not split). */
int gemm_strided_batched_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                            int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB, void *C,
                            int64_t ldc, int64_t strideC, int64_t batch, int dtype, void *stream);

/*
 * gemm_grouped -- `groups` independent products of different heights: problem g
 * uses the first m_g rows of A + g*strideA and C + g*strideC, and B + g*strideB,
 *     C_g[0:m_g, :] := A_g[0:m_g, :] . B_g,
 * where m_g = min(max(rows[g], 0), M).  This is the mixture-of-experts slice of
 * the Intel XPU Triton README (section "Use Tensor Descriptors to load tl.dot
 * arguments and save results", its A[expert, :tokens, :] example): each
 * expert's token count is read from device memory by the kernels, workgroups
 * whose tile starts at or past m_g exit early, and rows past m_g are masked.
 *   M         : the largest row count a problem may have (the row capacity of
 *               every A_g and C_g); sizes and strides are validated against it.
 *   rows      : DEVICE pointer to `groups` int32 counts, 4-byte aligned, read in
 *               stream order (a kernel earlier on `stream` may produce them).
 *               Values outside [0, M] are clamped, never an error: the host
 *               cannot see them.  Must be non-NULL when M, N and groups are > 0.
 *   Rows m_g .. M-1 of every C_g are not written.  Other arguments and rules as
 *   for gemm_strided_batched_ex (groups plays the role of batch).
 */
int gemm_grouped(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a, int64_t strideA,
                 const void *B, int64_t ldb, int layout_b, int64_t strideB, void *C, int64_t ldc, int64_t strideC,
                 const int32_t *rows, int64_t groups, int dtype, void *stream);

/* Element format of a row-sum input.  Sums are always float32. */
#define TSM_ROWSUM_F32 0
#define TSM_ROWSUM_F16 1
#define TSM_ROWSUM_BF16 2

/*
 * rowsum -- out[r] := sum_c X[r*row_stride + c*col_stride], r < R, c < C.
 * The tiled row-sum kernel of "A Dumb Triton Runtime Error" (sections "The
 * kernel itself" through "Step 3: Cross-Lane Tree Reduction (tl.sum) and Scalar
 * Store"): each element is converted to float32 and added into lane-local
 * float32 accumulators, tiles past the row end contribute 0, and one
 * cross-lane reduction per row is followed by one plain store.
 *   R, C        : rows and columns, >= 0.  C = 0 writes zeros.
 *   X           : device pointer, aligned to its element size (TSM_ROWSUM_*).
 *   row_stride,
 *   col_stride  : element strides, >= 0 (any view: transposed, sliced).
 *   out         : device float32 array of R sums, 4-byte aligned, OVERWRITTEN
 *                 (its previous contents never matter: "Making It Compile, and
 *                 Why I'd Still Use the Original").  Must not overlap X.
 * Accuracy: |out[r] - exact| <= C * 2^-24 * sum_c |X[r][c]|.  The reduction
 * order is fixed, so results are bitwise reproducible.
 * Errors and stream semantics as for gemm.
 */
int rowsum(int64_t R, int64_t C, const void *X, int64_t row_stride, int64_t col_stride, int xdtype, float *out,
           void *stream);

/* tsm_rowsum_kernel_name -- the kernel a rowsum call would launch, or NULL. */
const char *tsm_rowsum_kernel_name(int64_t R, int64_t C, const void *X, int64_t row_stride, int64_t col_stride,
                                   int xdtype, const float *out);

/*
 * gemm_strided_batched_act -- gemm_strided_batched_ex with an elementwise
 * activation fused into the epilogue: C := act(A.B), act applied to each
 * float32 result before it is converted and stored.  The ACTIVATION
 * meta-parameter of the Intel XPU Triton README's matmul signature ("Use
 * Proper Type Annotations") names such a fused activation; the pages do not
 * say which, so the plainest piecewise-linear ones are offered.
 *   activation: TSM_ACT_NONE, TSM_ACT_RELU or TSM_ACT_LEAKY_RELU.
 *   slope     : the factor leaky ReLU applies to negative values (finite);
 *               ignored otherwise.
 * Other arguments and rules as for gemm_strided_batched_ex.
 */
int gemm_strided_batched_act(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                             int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB, void *C,
                             int64_t ldc, int64_t strideC, int64_t batch, int dtype, int activation, float slope,
                             void *stream);

/*
 * gemm_workspace_bytes -- bytes of workspace with which gemm_strided_batched_ws
 * splits K for a problem of this shape: batch * S * M * N * 4 for S chunks of
 * K (the largest S the operands' layouts may lead to), or for the hybrid
 * r * s * 256 * 256 * 4 (see gemm_strided_batched_ws), or 0 when the shape
 * does not split (its output tiles already occupy the chip, K is below 512 or
 * not a multiple of 64, or N is not a multiple of 64 or 8).  With stream-K
 * requested (TSM_GEMM_SPLIT=streamk in the environment), also its need when
 * larger: 2 * R * 256 * 256 * 4 bytes for R runs (R = the CU count of the
 * current device, at most 256: 128 MiB).  Depends on the sizes (and then the
 * CU count) only.  Negative sizes give 0.
 */
int64_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t batch);

/*
 * gemm_strided_batched_ws -- gemm_strided_batched_act that may split K through
 * a caller's workspace, for products with few output tiles and deep K (e.g.
 * 256 x 256 x 8192, sixteen 64 x 64 tiles for 256 CUs).  The two-pass,
 * deterministic form of the split: pass 1 gives each workgroup one output tile
 * and one K chunk of 512 or more and stores its float32 partial sums into the
 * workspace; pass 2 adds the chunks of every output element in a fixed order,
 * applies the activation and the output conversion, and stores C once.  No
 * atomics, no zeroed memory: the store-once rule of "A Dumb Triton Runtime
 * Error" (section "The Takeaway and the Final Fix") holds across the split.
 *   workspace       : device memory owned by the caller, 16-byte aligned, not
 *                     overlapping A, B or C; its contents on entry do not
 *                     matter and on return are unspecified.  May be NULL
 *                     (with workspace_bytes = 0): the call then never splits.
 *   workspace_bytes : its size.  Below gemm_workspace_bytes(M, N, K, batch),
 *                     or for operands the split passes cannot read, the call
 *                     runs exactly as gemm_strided_batched_act.  The split
 *                     needs 16-byte aligned bases and rows (lda, ldb multiples
 *                     of 8, ldc of 4) and no grouped counts.  The streaming
 *                     kernel's split (up to 512 rows) needs row-major A, B
 *                     either way; the 256 x 256 tiles' split (above 128 rows,
 *                     one problem) takes any layout.
 * One problem of more than 256 tiles of 256 x 256 whose last round of 256 tiles
 * is at most half full (more than 128 rows, K a multiple of 128 from 2048 up)
 * takes the hybrid: the whole rounds run unsplit, and each of the r leftover
 * tiles is cut into s equal chunks of K (s r <= 256), whose float32 partial
 * tiles go to the workspace (r s * 256 * 256 * 4 bytes, at most 64 MiB) and
 * are added in K order before C is stored once.  Where row bands (see
 * gemm_strided_batched_ex) also apply, the hybrid is taken only for K above
 * 4096 with more than 64 rows past the whole rounds; TSM_GEMM_SPLIT=hybrid in
 * the environment takes it wherever it applies.
 * With TSM_GEMM_SPLIT=streamk in the environment, stream-K (the work-centric
 * decomposition of Osama et al., PPoPP 2023) replaces the tile split for 32
 * to 224 tiles of 256 x 256 (one problem or a strided batch, more than 128
 * rows, K a multiple of 128 from 2048 up): R workgroups, one per CU, take
 * equal runs of 128-deep slices of the tiles in order; every run meets at
 * most two tiles and stores a float32 partial tile for each into the
 * workspace, and a second kernel adds each tile's partials in K order and
 * stores C once.  The result is the same on every call on devices with the
 * same CU count.  It is not the default: on MI355X it is slower than the
 * plain kernel or the tile split for these shapes.  TSM_GEMM_SPLIT=none
 * keeps the kernel that needs no workspace.
 * Two calls in flight at once must not share a workspace.  Other arguments,
 * rules and errors as for gemm_strided_batched_act; additionally
 * TSM_ERROR_INVALID_VALUE for negative workspace_bytes, a NULL workspace with
 * workspace_bytes > 0, a misaligned workspace or one overlapping an operand.
 */
int gemm_strided_batched_ws(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                            int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB, void *C,
                            int64_t ldc, int64_t strideC, int64_t batch, int dtype, int activation, float slope,
                            void *workspace, int64_t workspace_bytes, void *stream);

/*
 * gemm_strided_batched_noalloc -- gemm_strided_batched_ws for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation): the K split's partial sums go to a
 * static scratch array of gemm_noalloc_scratch_bytes() (64 MiB) that the
 * library holds on each GPU from its load until the process ends.  The call
 * allocates nothing.  It splits K exactly when gemm_strided_batched_ws would
 * with a workspace of gemm_workspace_bytes(M, N, K, batch) bytes; shapes that
 * do not split run as gemm_strided_batched_act.
 * Calls on one GPU share its scratch: calls that overlap on one GPU (other
 * streams, other host threads) race and must not be issued.  The scratch
 * needs no clearing (every partial read back was written by the same call).
 * Arguments and errors as for gemm_strided_batched_act; additionally
 * TSM_ERROR_NOT_SUPPORTED when the split would need more than the scratch
 * holds (the detail names the size; use gemm_strided_batched_ws then), and
 * TSM_ERROR_LAUNCH when the scratch's device address cannot be obtained.
 */
int gemm_strided_batched_noalloc(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                                 int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB, void *C,
                                 int64_t ldc, int64_t strideC, int64_t batch, int dtype, int activation, float slope,
                                 void *stream);

/* Bytes of the static scratch gemm_strided_batched_noalloc splits K through. */
int64_t gemm_noalloc_scratch_bytes(void);

/* ---- Int8 products and expert routing ------------------------------------------
 * Element formats of the entry points below (f32, f16 and bf16 as TSM_ROWSUM_*),
 * and the integer formats of expert ids. */
#define TSM_F32 0
#define TSM_F16 1
#define TSM_BF16 2
#define TSM_I8 3
#define TSM_I32 4
#define TSM_I64 5

/*
 * quantize_i8 -- rows to int8 codes with one float32 scale each, for gemm_i8:
 * with m the largest magnitude of row r,
 *     scale[r] := m / 127,    Q[r][c] := nearest whole number to 127 X[r][c] / m,
 * ties to even, so X[r][c] is Q[r][c] * scale[r] to within half a step.  The
 * codes are those of the exact quotient (no intermediate rounding).  A row of
 * zeros gets scale 0 and codes 0; a row that holds a NaN or an infinity gets
 * scale NaN and codes 0, so every product with it is NaN.  (A scale below the
 * normal float32 range, of an m below 127 * 2^-126, is rounded to that range's
 * steps, and X then differs by as much more.)
 *   R, C       : rows and columns per group, >= 0.  C = 0 writes scales of 0.
 *   X, ldx     : X[g*strideX + r*ldx + c], format xdtype (TSM_F32, TSM_F16 or
 *                TSM_BF16), aligned to its element; ldx >= 0 (rows may overlap
 *                or repeat).
 *   Q, ldq     : codes, ldq >= C; padding is not written.
 *   scale      : scale[g*stride_scale + r], stride_scale >= R for several groups.
 *   rows       : NULL, or a DEVICE array of `groups` int32 counts as gemm_grouped
 *                takes them: rows at and past rows[g] are neither read nor written.
 *   groups     : matrices (1 for a single one, whose strides are ignored).
 * Errors and stream semantics as for gemm; Q and scale must not overlap X or
 * each other.
 */
int quantize_i8(int64_t R, int64_t C, const void *X, int64_t ldx, int64_t strideX, int xdtype, int8_t *Q, int64_t ldq,
                int64_t strideQ, float *scale, int64_t stride_scale, const int32_t *rows, int64_t groups,
                void *stream);

/*
 * gemm_i8 -- product of int8 codes with a scale for each token (row of A) and
 * each channel (column of B):
 *     C[i][j] := scale_a[i] * scale_b[j] * sum_k A[i][k] * B[j*ldb + k].
 * The sum is an exact int32 (so K <= 131071); it is converted to float32 once,
 * multiplied by scale_a, then by scale_b, and rounded to the output format.
 *   A, lda     : codes, row-major M x K, lda >= K, any alignment.
 *   B, ldb     : codes of the weight stored N x K (column-major B), ldb >= K.
 *   scale_a/_b : device float32, M and N of them; NULL means ones.
 *   C, ldc     : row-major result, out_dtype TSM_F32, TSM_F16 or TSM_BF16.
 * K = 0 gives sums of 0 (times the scales).  Errors and stream semantics as for
 * gemm; C must not overlap an operand or a scale.
 */
int gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a, const int8_t *B,
            int64_t ldb, const float *scale_b, void *C, int64_t ldc, int out_dtype, void *stream);

/*
 * gemm_i8_strided_batched -- `batch` such products at element strides (0 shares
 * an operand or its scales; strideC keeps the outputs disjoint), with the fused
 * activation of gemm_strided_batched_act applied after the scales.  A NaN (of a
 * scale) stays NaN with every activation; the 16-bit products' ReLU gives 0.
 */
int gemm_i8_strided_batched(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                            const float *scale_a, int64_t stride_sa, const int8_t *B, int64_t ldb, int64_t strideB,
                            const float *scale_b, int64_t stride_sb, void *C, int64_t ldc, int64_t strideC,
                            int64_t batch, int out_dtype, int activation, float slope, void *stream);

/*
 * gemm_i8_grouped -- the same over a mixture of experts' slabs: problem g uses
 * its first m_g = min(max(rows[g], 0), M) rows, counts in device memory, as
 * gemm_grouped.  Rows past m_g of A, scale_a and C are neither read nor written.
 */
int gemm_i8_grouped(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                    const float *scale_a, int64_t stride_sa, const int8_t *B, int64_t ldb, int64_t strideB,
                    const float *scale_b, int64_t stride_sb, void *C, int64_t ldc, int64_t strideC,
                    const int32_t *rows, int64_t groups, int out_dtype, int activation, float slope, void *stream);

/* tsm_gemm_i8_kernel_name -- the kernel a gemm_i8_strided_batched call (rows NULL)
 * or a gemm_i8_grouped call would launch, or NULL. */
const char *tsm_gemm_i8_kernel_name(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, int64_t strideA,
                                    const int8_t *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                                    int64_t strideC, int64_t batch, const int32_t *rows, int out_dtype);

/*
 * moe_sort -- the row of each (token, choice) in its expert's slab.  The slabs
 * of all experts are one matrix of experts * capacity rows, expert e's from row
 * e * capacity (what gemm_grouped and gemm_i8_grouped take with
 * strideA = capacity * lda).  With e = ids[t*ld_ids + j],
 *     positions[t*topk + j] := e * capacity + r,
 * r the number of entries before (t, j), in token order, that chose e; -1 when
 * e is outside [0, experts) (a padded token) or r >= capacity (dropped).
 *     counts[e] := all entries that chose e (those past capacity among them;
 * the grouped products clamp to their M).
 *   ids        : DEVICE expert ids, idtype TSM_I32 or TSM_I64, ld_ids >= topk.
 *   experts    : at most 512.  experts * capacity and tokens * topk below 2^31.
 *   workspace  : DEVICE memory of moe_sort_workspace_bytes(...) bytes, 16-byte
 *                aligned, its contents irrelevant before and after (NULL where
 *                that is 0).  Calls in flight at once must not share one.
 * The result is the same on every call.  tokens = 0 or topk = 0 writes counts of 0.
 */
int moe_sort(int64_t tokens, int64_t topk, const void *ids, int64_t ld_ids, int idtype, int64_t experts,
             int64_t capacity, int32_t *positions, int32_t *counts, void *workspace, int64_t workspace_bytes,
             void *stream);
int64_t moe_sort_workspace_bytes(int64_t tokens, int64_t topk, int64_t experts);

/*
 * moe_dispatch -- slabs[positions[t*topk + j]] := X[t], and slab_scale likewise
 * from scale, for every entry with a position.  Slab rows without an entry keep
 * what they held.  Positions at or past `slots` count as none; no two entries
 * may have the same one (moe_sort gives distinct ones).
 *   X, ldx     : tokens x hidden, dtype TSM_F32, TSM_F16, TSM_BF16 or TSM_I8.
 *   slabs      : slots x hidden, ld_slabs >= hidden.
 *   scale, slab_scale : a float32 per token and per slab row (the scales of
 *                quantize_i8), or both NULL.
 * Its gradient is moe_combine with weights NULL.
 */
int moe_dispatch(int64_t tokens, int64_t topk, int64_t hidden, const void *X, int64_t ldx, int dtype,
                 const float *scale, const int32_t *positions, int64_t slots, void *slabs, int64_t ld_slabs,
                 float *slab_scale, void *stream);

/*
 * moe_combine -- Y[t] := sum_j weights[t*topk + j] * slabs[positions[t*topk + j]],
 * over the entries with a position (no others count: a NaN weight of one without
 * a position or a stale slab row does not matter); float32 sums in
 * the order of j, rounded once.  weights NULL means ones.  A token without any
 * gets zeros.  dtype (slabs and Y): TSM_F32, TSM_F16 or TSM_BF16.
 */
int moe_combine(int64_t tokens, int64_t topk, int64_t hidden, const void *slabs, int64_t ld_slabs, int64_t slots,
                int dtype, const int32_t *positions, const float *weights, void *Y, int64_t ldy, void *stream);

/*
 * moe_combine_backward -- the gradients of moe_combine from dY (tokens x hidden):
 *     dslabs[positions[t*topk + j]]  := weights[t*topk + j] * dY[t],
 *     dweights[t*topk + j]           := <dY[t], slabs[positions[t*topk + j]]>,
 * float32 sums; dweights is 0 where there is no position, and dslabs rows
 * without an entry keep what they held.  dslabs must not overlap slabs.
 */
int moe_combine_backward(int64_t tokens, int64_t topk, int64_t hidden, const void *dY, int64_t lddy, const void *slabs,
                         int64_t ld_slabs, int64_t slots, int dtype, const int32_t *positions, const float *weights,
                         void *dslabs, int64_t ld_dslabs, float *dweights, void *stream);

/* ---- Microscaled 4-bit products --------------------------------------------------
 * A row of C elements in microscaled 4-bit form (mx4: the MXFP4 of the OCP
 * Microscaling Formats specification) is
 *   codes  : (C + 1) / 2 bytes, element 2i in the low half of byte i and 2i + 1 in
 *            the high half: bit 3 the sign, bits 0..2 one of 0, 0.5, 1, 1.5, 2, 3,
 *            4, 6.  The last high half of an odd C is 0 and is never looked at.
 *   scales : (C + 31) / 32 bytes, one per block of 32 elements: E stands for
 *            2^(E - 127), and 255 for a block of NaN whatever its codes.
 * Leading dimensions and strides of codes and scales are in bytes; neither needs
 * any alignment.  The fast kernels of the products need all three: K a multiple of
 * 128, rows of codes at multiples of 16 bytes, rows of scales at multiples of 4;
 * every other product runs on the general kernels (mx4_block_*).
 *
 * mx4_quantize -- rows to that form: of each block's largest magnitude m
 *     E := max(0, 127 + floor(log2 m) - 2),   code := nearest to |X| / 2^(E - 127),
 * ties to the even code, magnitudes above 6 (m up to 8 scales) to 6.  A block of
 * zeros gets E = 0; one that holds a NaN or an infinity E = 255 and codes of 0, so
 * every product with it is NaN.
 *   R, C       : rows and elements per row, of each of `groups` matrices.
 *   layout     : TSM_ROW: X[g*strideX + r*ldx + c]; TSM_COL: X[g*strideX + c*ldx + r]
 *                (blocks along the rows of the stored matrix: the operands of a
 *                weight gradient).  Format xdtype (TSM_F32, TSM_F16 or TSM_BF16).
 *   rows       : NULL, or a DEVICE array of `groups` int32 counts: rows at and past
 *                rows[g] are neither read nor written.
 * Errors and stream semantics as for quantize_i8.
 */
int mx4_quantize(int64_t R, int64_t C, const void *X, int64_t ldx, int layout, int64_t strideX, int xdtype, uint8_t *Q,
                 int64_t ldq, int64_t strideQ, uint8_t *scale, int64_t ld_scale, int64_t stride_scale,
                 const int32_t *rows, int64_t groups, void *stream);

/* mx4_dequantize -- the values of codes and scales, Y[g*strideY + r*ldy + c], each
 * rounded once to ydtype (to infinity where it is too large for that). */
int mx4_dequantize(int64_t R, int64_t C, const uint8_t *Q, int64_t ldq, int64_t strideQ, const uint8_t *scale,
                   int64_t ld_scale, int64_t stride_scale, void *Y, int64_t ldy, int64_t strideY, int ydtype,
                   const int32_t *rows, int64_t groups, void *stream);

/*
 * gemm_mx4 -- C[i][j] := sum_k A[i][k] * B[j][k] for operands in mx4 form, A of M
 * rows and B of N rows (a weight stored N x K) of K elements each.  Products of two
 * elements are exact, sums are float32; |C - exact| <= K * 2^-24 * sum |a b|, plus
 * the rounding to out_dtype (TSM_F32, TSM_F16 or TSM_BF16).  K = 0 gives zeros.
 * Errors and stream semantics as for gemm; C must not overlap an operand.
 */
int gemm_mx4(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *scale_a, int64_t ld_sa,
             const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ld_sb, void *C, int64_t ldc, int out_dtype,
             void *stream);

/* gemm_mx4_strided_batched, gemm_mx4_grouped -- as gemm_i8_strided_batched and
 * gemm_i8_grouped: `batch` products at strides (0 shares an operand), or experts'
 * slabs with row counts in device memory; an activation, in which a NaN stays one.
 * A grouped call's kernel is chosen by M, the rows of a slab, since its counts are
 * known on the GPU only: slabs of thousands of rows run on large tiles however few
 * of them are filled. */
int gemm_mx4_strided_batched(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                             const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B, int64_t ldb,
                             int64_t strideB, const uint8_t *scale_b, int64_t ld_sb, int64_t stride_sb, void *C,
                             int64_t ldc, int64_t strideC, int64_t batch, int out_dtype, int activation, float slope,
                             void *stream);
int gemm_mx4_grouped(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                     const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B, int64_t ldb,
                     int64_t strideB, const uint8_t *scale_b, int64_t ld_sb, int64_t stride_sb, void *C, int64_t ldc,
                     int64_t strideC, const int32_t *rows, int64_t groups, int out_dtype, int activation, float slope,
                     void *stream);

/*
 * gemm_mx4_float_a -- mx4_quantize of activations X (TSM_ROW, format xdtype) and
 * their product with B in one call: the codes and scales of mx4_quantize; the
 * kernel, and with it the order of the sums, may be another than gemm_mx4's.
 *   rows      : NULL (a strided batch, strideX = 0 shares X), or counts as
 *               gemm_mx4_grouped takes them.
 *   workspace : DEVICE memory of gemm_mx4_float_a_workspace_bytes(M, K, batch)
 *               bytes (with strideX = 0, of batch 1), 16-byte aligned, overlapping
 *               nothing else, its contents irrelevant before and after.  Calls in
 *               flight at once must not share one.
 */
int gemm_mx4_float_a(int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx, int64_t strideX, int xdtype,
                     const uint8_t *B, int64_t ldb, int64_t strideB, const uint8_t *scale_b, int64_t ld_sb,
                     int64_t stride_sb, void *C, int64_t ldc, int64_t strideC, int64_t batch, const int32_t *rows,
                     int out_dtype, int activation, float slope, void *workspace, int64_t workspace_bytes,
                     void *stream);
int64_t gemm_mx4_float_a_workspace_bytes(int64_t M, int64_t K, int64_t batch);

/* tsm_gemm_mx4_kernel_name -- the kernel a gemm_mx4_strided_batched call (rows
 * NULL) or a gemm_mx4_grouped call would launch, or NULL.  A gemm_mx4_float_a call
 * launches the same behind its quantisation, but for one or two rows that mx4_stream
 * would multiply: those are quantised within the launch of a kernel of its own, which
 * has no name here (TSM_GEMM_KERNEL=mx4_stream keeps to the two launches). */
const char *tsm_gemm_mx4_kernel_name(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, int64_t strideA,
                                     const uint8_t *scale_a, int64_t ld_sa, int64_t stride_sa, const uint8_t *B,
                                     int64_t ldb, int64_t strideB, const uint8_t *scale_b, int64_t ld_sb,
                                     int64_t stride_sb, void *C, int64_t ldc, int64_t strideC, int64_t batch,
                                     const int32_t *rows, int out_dtype);

/* ---- Expert router --------------------------------------------------------------- */
#define TSM_SCORE_SOFTMAX 0
#define TSM_SCORE_SIGMOID 1

/*
 * moe_route -- each token's experts and their weights, from the router's logits
 * x (tokens x experts, format TSM_F32, TSM_F16 or TSM_BF16):
 *   scores  : s_e = exp(x_e) / sum exp(x), or 1 / (1 + exp(-x_e)).
 *   bias    : NULL, or a DEVICE float32 per expert, added to the scores to choose
 *             (the key s_e + bias_e) and not to weigh (a bias for balance).
 *   groups  : the experts stand in `groups` groups of equal size, one after another;
 *             only those of the top_groups groups are chosen from whose group_best
 *             (1 or 2) largest keys have the largest sum.  top_groups = groups: from all.
 *   ids     : the topk experts of the largest keys, in that order (what moe_sort takes).
 *   weights : factor * s_e, or with renormalize factor * s_e over the sum of the
 *             chosen experts' s (finite, however small those are).
 * Equal keys (and sums) go to the lowest index.  The choice is the one of exact
 * scores, up to differences of keys below 2^-50 (of keys past 1, 2^-50 of them).  An expert whose logit (or bias) is -inf
 * or NaN is never chosen, and where none is left the id is -1 and the weight 0: a
 * padded token with a row of -inf gets no expert.  A row with a NaN (or, for a
 * softmax, +inf) among its logits gets weights of NaN; its ids are those of its
 * largest logits, whatever the bias and the groups.
 * experts at most 512, topk and the groups to choose from at most 64, topk at most
 * the experts of top_groups groups.  ids and weights are tokens x topk, packed.
 */
int moe_route(int64_t tokens, int64_t experts, int64_t topk, const void *logits, int64_t ld_logits, int dtype,
              int scores, const float *bias, int64_t groups, int64_t top_groups, int group_best, int renormalize,
              float factor, int32_t *ids, float *weights, void *stream);

/*
 * moe_route_backward -- the gradient of the logits from that of the weights, for
 * chosen ids (which, and with them the bias, take no gradient):
 *     dlogits[t][e] := sum_j dweights[t][j] * d weights[t][j] / d x_e,
 * float32 sums, rounded once to the logits' format.  Ids outside [0, experts) have
 * no weight; an id may occur more than once in a token's row.  An expert of logit
 * -inf gets 0.  dlogits is written whole and must not overlap an input.
 */
int moe_route_backward(int64_t tokens, int64_t experts, int64_t topk, const float *dweights, const void *logits,
                       int64_t ld_logits, int dtype, const int32_t *ids, int scores, int renormalize, float factor,
                       void *dlogits, int64_t ld_dlogits, void *stream);

/* Static text for a status code ("success", "invalid value", ...). */
const char *tsm_status_string(int status);

/* Text naming the check that made the calling thread's last call fail
 * (thread-local; empty after a successful call). */
const char *tsm_last_error_detail(void);

/*
 * tsm_gemm_kernel_name -- name of the kernel variant a gemm_strided_batched_ex
 * call with these arguments would launch (same arguments, no stream), or NULL
 * if the call would be rejected or launch nothing.  Pure host logic: it
 * validates and selects, it never touches the GPU.  The returned string is
 * static.
 */
const char *tsm_gemm_kernel_name(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                                 int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB,
                                 void *C, int64_t ldc, int64_t strideC, int64_t batch, int dtype);

/* tsm_gemm_ws_kernel_name -- the same for a gemm_strided_batched_ws call (a
 * split names its pass-1 kernel followed by "+reduce"). */
const char *tsm_gemm_ws_kernel_name(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                                    int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB,
                                    void *C, int64_t ldc, int64_t strideC, int64_t batch, int dtype,
                                    const void *workspace, int64_t workspace_bytes);

/* tsm_gemm_grouped_kernel_name -- the same for a gemm_grouped call. */
const char *tsm_gemm_grouped_kernel_name(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int layout_a,
                                         int64_t strideA, const void *B, int64_t ldb, int layout_b, int64_t strideB,
                                         void *C, int64_t ldc, int64_t strideC, const int32_t *rows, int64_t groups,
                                         int dtype);

#ifdef __cplusplus
}
#endif

#endif /* TSM_GEMM_H */
