/*
 * gemm_epi_experts.h -- the feed-forward of a mixture of experts and products
 * of 8-bit integers: the router, products grouped by expert, the combination
 * of a token's rows, the quantisation of rows, and the product of such rows
 * with 8-bit weights.
 *
 * Plain C, like gemm_epi.h, whose formats, status codes and manners they
 * share: device buffers are plain device pointers owned by the caller, the
 * stream is a hipStream_t passed as void* (NULL = the null stream) of the
 * current device, every call validates its arguments on the host, enqueues
 * on the stream and returns without synchronising, allocates nothing, needs
 * no workspace, and can be captured into a graph.  A leading dimension is the
 * number of elements between consecutive rows.  The same inputs give the same
 * bits.  Forward only, as the rest of the library.
 *
 * A layer of experts for `tokens` rows x of which each goes to `per` experts:
 *     gemm_epi_route          logits -> ids, weights, offsets, order
 *     gemm_epi_grouped_gemm   h = silu(x Wg^T) * (x Wu^T), rows gathered
 *     gemm_epi_grouped_gemm   z = h Wd^T, rows scattered to their entries
 *     gemm_epi_combine        y = r + sum of a token's z, weighted
 * An entry is a token's j-th choice, number t * per + j.
 */
#ifndef GEMM_EPI_EXPERTS_H
#define GEMM_EPI_EXPERTS_H

#include "gemm_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* gemm_epi_quantise_i8 -- rows in 8-bit integers with a scale each,
 *
 *     scale = max(max_j |x_j| / 127, 2^-100)        y_j = x_j / scale
 *
 * the quotients in fp32, y_j rounded to the nearest integer (ties to even).
 *   X      rows x cols (ldx), format `dtype` (F16 or BF16)
 *   Y      rows x cols (ldy), 8-bit integers
 *   scale  rows fp32 values
 * A row that holds an infinity or a NaN gets scale NaN and zeros (all its
 * values read as NaN, and its products are NaN, of which a ReLU, max(z, 0),
 * makes 0).  Y and scale overlap nothing else.  Any alignment of an
 * element.  rows = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer, rows < 0, cols <= 0, a leading
 * dimension below cols, dtype not F16 or BF16, a pointer off its element's
 * alignment), UNSUPPORTED (rows >= 2^31, cols above 2^30), HIP. */
gemm_epi_status gemm_epi_quantise_i8(const void* X, int64_t ldx, int8_t* Y, int64_t ldy, float* scale, int64_t rows,
                                     int64_t cols, gemm_epi_dtype dtype, void* stream);

/* gemm_epi_i8_gemm -- product of 8-bit integers with a scale for each row of
 * A (a token) and each column (a channel of the weights),
 *
 *     C = act((A B^T) a_scale[m] b_scale[n] + bias[n]) + R
 *
 *   A   M x K (lda), 8-bit integers     a_scale  M fp32 values
 *   B   N x K (ldb), 8-bit integers     b_scale  N fp32 values
 *   bias  N values of out_dtype, for an epilogue with one (else ignored)
 *   R   M x N (ldr), out_dtype, or NULL
 *   C   M x N (ldc), out_dtype: F16 or BF16
 * The sum over k is exact (32-bit integers), the rest is fp32 in the order
 * written, rounded once.  R may be C itself (same pointer and leading
 * dimension); nothing else may overlap C.  M = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer where one is needed, M < 0, N or K <= 0,
 * a leading dimension below its row, an unknown epilogue, out_dtype not F16 or
 * BF16, a pointer off its element's alignment), UNSUPPORTED (K not a multiple
 * of 16 or >= 2^17, A or B not 16-byte aligned, lda or ldb not a multiple of
 * 16 or above 2^24, any size or leading dimension >= 2^31, more than 2^25
 * blocks of 16 x 16 outputs), HIP. */
gemm_epi_status gemm_epi_i8_gemm(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                                 const float* b_scale, const void* bias, const void* R, int64_t ldr, void* C,
                                 int64_t ldc, int64_t M, int64_t N, int64_t K, gemm_epi_epilogue epilogue,
                                 gemm_epi_dtype out_dtype, void* stream);

/* How logits become weights: over all experts, or each for itself. */
typedef enum gemm_epi_score { GEMM_EPI_SOFTMAX = 0, GEMM_EPI_SIGMOID = 1 } gemm_epi_score;

/* gemm_epi_route -- the experts of each token, and all entries in their order.
 *
 *   logits   tokens x experts (ldl), format `dtype`: F32, F16 or BF16
 *   ids      tokens x per: the experts of the `per` largest logits, in
 *            descending order, of equal ones the lower expert first
 *   weights  tokens x per fp32: p_j * scale with p = softmax of the token's
 *            logits or 1 / (1 + exp(-logit)); with renormalise, p is divided
 *            by its sum over the chosen experts
 *   offsets, order  as gemm_epi_group_rows writes them for these ids, or NULL
 *            both
 * A NaN counts as minus infinity, and an expert at minus infinity is not
 * chosen: where too few are left, id -1 and weight 0.  The softmax of plus
 * infinities is shared evenly among them.
 * tokens = 0 chooses nothing; offsets are then zeros.
 * Errors: INVALID_ARG (a NULL pointer where one is needed, one of offsets and
 * order without the other, tokens < 0, experts or per <= 0, per > experts, ldl
 * below experts, an unknown score, a scale that is not finite, dtype not F32,
 * F16 or BF16, a pointer off its element's alignment), UNSUPPORTED (more than
 * 1024 experts, per above 64, more than 2^25 tokens, tokens * per or ldl >=
 * 2^31), HIP. */
gemm_epi_status gemm_epi_route(const void* logits, int64_t ldl, gemm_epi_dtype dtype, int64_t tokens, int64_t experts,
                               int64_t per, gemm_epi_score score, int renormalise, float scale, int32_t* ids,
                               float* weights, int32_t* offsets, int32_t* order, void* stream);

/* gemm_epi_group_rows -- the entries by group, stable.
 *   ids      rows values; outside [0, groups): an entry of no group
 *   offsets  groups + 1: where each group begins in `order`
 *   order    rows: the entries' numbers, group by group, ascending in each;
 *            -1 from offsets[groups] on
 * Errors: INVALID_ARG (a NULL pointer where one is needed, rows < 0, groups <=
 * 0, a pointer off its alignment), UNSUPPORTED (more than 1024 groups, rows >=
 * 2^31), HIP. */
gemm_epi_status gemm_epi_group_rows(const int32_t* ids, int64_t rows, int64_t groups, int32_t* offsets, int32_t* order,
                                    void* stream);

/* The rows of a grouped product.  Place i of [offsets[g], offsets[g + 1])
 * belongs to group g and is entry q = order[i] (order NULL: q = i).  Both arrays
 * are in device memory and are read when the kernel runs, so a captured graph
 * follows what they hold at its replay.  Offsets are taken as clamped to [0,
 * rows] and as no lower than any before them, so that no place is of two groups;
 * an order outside [0, rows) is no entry. */
typedef struct gemm_epi_groups {
  const int32_t* offsets; /* [groups + 1] */
  const int32_t* order;   /* [rows] or NULL */
  int64_t groups;
  int64_t rows; /* places there are at most */
  int64_t per;  /* entries of a row of a gathered X */
} gemm_epi_groups;

#define GEMM_EPI_GATHER 1  /* X has rows / per rows, entry q reads row q / per; else place i reads row i of `rows` */
#define GEMM_EPI_SCATTER 2 /* entry q writes row q of C; else place i writes row i */
#define GEMM_EPI_GATED 4   /* C = act(gate) * up */

/* gemm_epi_grouped_gemm -- products grouped by expert: for place i of group g
 *
 *     C[.] = act(X[.] W[g]^T + bias[g])
 *     C[.] = act(X[.] W[g]^T + bias[g]) * (X[.] V[g]^T + bias'[g])     GATED
 *
 *   X   rows of K values (ldx), format `dtype`: F16, BF16 or I8
 *   W   groups x N x K packed; GATED: groups x 2 N x K, V[g] behind W[g]
 *   bias  groups x N (2 N) of out_dtype, for an epilogue with one (else ignored)
 *   x_scale, w_scale  I8 only: a fp32 factor for each row of X, and for each
 *       row of W (groups x N, or 2 N), as in gemm_epi_i8_gemm
 *   C   rows of N values (ldc), out_dtype: `dtype`, or F16 or BF16 for I8
 * Sums in fp32 (I8: exact), one rounding.  Rows of C that no place writes are
 * left as they were.  C overlaps nothing else.  An entry that occurs twice is
 * written twice, with which of both values is not defined.  rows = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer where one is needed, rows < 0, groups, per,
 * N or K <= 0, a leading dimension below its row, unknown flags or epilogue,
 * formats that do not fit, scales missing or not wanted, SCATTER or GATHER
 * without order, rows not a multiple of per with GATHER, a pointer off its
 * element's alignment), UNSUPPORTED (rows of K not a multiple of 16 bytes, K >=
 * 2^17, X or W not 16-byte aligned, ldx not a multiple of 16 bytes or above 16
 * MiB, more than 1024 groups, any size or leading dimension >= 2^31, X of 4 GiB
 * less 64 KiB or more with GATHER, gates of a group of more than 2 GiB, more
 * than 2^25 blocks of 16 x 16 products, counting one more for each group),
 * HIP. */
gemm_epi_status gemm_epi_grouped_gemm(const gemm_epi_groups* groups, const void* X, int64_t ldx, const float* x_scale,
                                      const void* W, const float* w_scale, const void* bias, void* C, int64_t ldc,
                                      int64_t N, int64_t K, int flags, gemm_epi_epilogue epilogue,
                                      gemm_epi_dtype dtype, gemm_epi_dtype out_dtype, void* stream);

/* gemm_epi_combine -- the rows of each token's entries, weighted,
 *
 *     Y[t] = R[t] + sum_j weights[t, j] Z[t per + j]     over the j with 0 <= ids[t, j] < experts
 *
 * in fp32, rounded once (the sum over j first, in ascending order).
 *   Z   tokens * per rows of cols (ldz), format `dtype`: F16 or BF16
 *   weights  tokens x per fp32
 *   ids  tokens x per, or NULL: all take part.  The row of an entry of no
 *        expert is not read.
 *   R   tokens x cols (ldr), `dtype`, or NULL
 *   Y   tokens x cols (ldy), `dtype`; may be R itself (same pointer and
 *       leading dimension); overlaps nothing else
 * Any alignment of an element.  tokens = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer where one is needed, tokens < 0, per,
 * cols or experts <= 0, a leading dimension below cols, dtype not F16 or BF16,
 * a pointer off its element's alignment), UNSUPPORTED (per above 64, tokens *
 * per >= 2^31, cols above 2^30), HIP. */
gemm_epi_status gemm_epi_combine(const void* Z, int64_t ldz, const float* weights, const int32_t* ids, int64_t experts,
                                 const void* R, int64_t ldr, void* Y, int64_t ldy, int64_t tokens, int64_t per,
                                 int64_t cols, gemm_epi_dtype dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_EXPERTS_H */
