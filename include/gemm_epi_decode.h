/*
 * gemm_epi_decode.h -- the operators that stand between the products of a
 * decode step: the RMS norm with the residual's addition, low-rank adapters
 * of many requests beside a shared projection, the paged key-value cache
 * and the attention of one new token over it.
 *
 * Plain C, like gemm_epi.h, whose formats, status codes and manners they
 * share: device buffers are plain device pointers owned by the caller, the
 * stream is a hipStream_t passed as void* (NULL = the null stream) of the
 * current device, every call validates its arguments on the host, enqueues
 * on the stream and returns without synchronising, allocates nothing, and
 * can be captured into a graph.  A leading dimension is the number of
 * elements between consecutive rows.  Forward only, as the rest of the
 * library.
 */
#ifndef GEMM_EPI_DECODE_H
#define GEMM_EPI_DECODE_H

#include "gemm_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* gemm_epi_rmsnorm -- root-mean-square norm with the residual's addition,
 *
 *     h = x + r            y = h / sqrt(mean(h^2) + eps) * w
 *
 * for each of `rows` rows of `cols` elements, in fp32, every output rounded
 * once (y from the unrounded h).
 *   X   rows x cols (ldx), format `dtype` (F16 or BF16)
 *   R   the residual, rows x cols (ldr), or NULL: h = x
 *   W   cols weights, format `dtype`
 *   H   receives h, rows x cols (ldh), format `dtype`, or NULL
 *   Y   receives y, rows x cols (ldy), format out_dtype: `dtype`, or FP8_E4M3
 *       with one scale per row in y_scale (rows fp32 values):
 *       y_scale = max(max_j |y_j| / 448, 2^-100), and Y holds y / y_scale
 *       rounded to nearest even
 *   y_scale  NULL unless out_dtype is FP8_E4M3
 * H and Y may each be X or R itself (same pointer and leading dimension; Y
 * only in format `dtype`); nothing else may overlap an output.
 * The sum of squares is an fp32 sum: a row holding an infinity or NaN, or
 * values whose squares overflow it, is normalised by that sum.  h w is an
 * fp32 product, formed before the division: where it overflows, so does y.
 * Any alignment of an element; 16-byte aligned pointers and leading
 * dimensions that are multiples of 8 take the fast path (W included).
 * rows = 0 does nothing.
 * Errors: INVALID_ARG (a NULL X, W or Y, rows < 0, cols <= 0, a leading
 * dimension below cols, eps negative or not finite, a format that is not
 * allowed, y_scale missing or not wanted, a pointer off its element's
 * alignment), UNSUPPORTED (rows or cols >= 2^31), HIP. */
gemm_epi_status gemm_epi_rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* W, void* H,
                                 int64_t ldh, void* Y, int64_t ldy, float* y_scale, int64_t rows, int64_t cols,
                                 float eps, gemm_epi_dtype dtype, gemm_epi_dtype out_dtype, void* stream);

/* gemm_epi_lora -- low-rank adapters of many requests at once,
 *
 *     C[m] = R[m] + s[a] (X[m] A[a]^T) B[a]^T        a = ids[m]
 *
 * beside the projection that all rows share.  With R = the projection's
 * output (in place: C = R), it adds the adapters to it; with R = NULL, C is
 * the adapters' part alone, to be given to gemm_epi_run_ex as the residual
 * of the projection (then rounded once with it).
 *   X   M x K (ldx), the projection's input     A   adapters x rank x K
 *   C   M x N (ldc)                             B   adapters x N x rank
 *   R   M x N (ldr) or NULL                     all of format `dtype` (F16, BF16)
 *   scale  one fp32 factor per adapter, or NULL for 1
 *   ids    M values: the adapter of each row, in any order; a value outside
 *          [0, adapters) is a row without one (C[m] = R[m], or 0)
 * A and B are packed.  R may be C itself (same pointer and leading
 * dimension); nothing else may overlap C or the workspace.  The inner
 * product X A^T is kept in fp32; it enters the second product as two
 * 16-bit parts of each row scaled by a power of two (16 significant bits in
 * BF16, 22 in F16); sums in fp32, one rounding.  What meets an infinity of B is
 * an infinity or NaN.
 * workspace: gemm_epi_lora_workspace_size bytes, 16-byte aligned, with no
 * content of its own before or after a call; calls that share it must not
 * overlap in time.
 * M = 0 does nothing.  The result of a row depends on that row, its adapter
 * and the problem's sizes only.
 * Errors: INVALID_ARG (a NULL pointer where one is needed, M < 0, N, K, rank
 * or adapters <= 0, a leading dimension below its row, dtype not F16/BF16,
 * workspace missing or too small, a pointer off its element's alignment),
 * UNSUPPORTED (rank above 128 or not a multiple of 8, K not a multiple of 8,
 * ldx not a multiple of 8, X, A, B or workspace not 16-byte aligned, M above
 * 2^28 - 16, K >= 2^28, N above 65535 * 256, more than 65535 adapters),
 * HIP. */
gemm_epi_status gemm_epi_lora(const void* X, int64_t ldx, const void* A, const void* B, const float* scale,
                              const int32_t* ids, const void* R, int64_t ldr, void* C, int64_t ldc, int64_t M,
                              int64_t N, int64_t K, int64_t rank, int64_t adapters, gemm_epi_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace gemm_epi_lora needs for these sizes (0 when it would
 * refuse them, or M = 0).  Host only. */
size_t gemm_epi_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters);

/* A paged key-value cache of one layer: num_pages pages of page_size tokens,
 * each page holding its tokens' rows head by head, so that a head's rows of
 * a page are contiguous.
 *   k, v              [num_pages, heads, page_size, head_dim], format `dtype`:
 *                     F16, BF16 or FP8_E4M3
 *   k_scale, v_scale  FP8_E4M3 only (else NULL): [num_pages, heads, page_size]
 *                     fp32, a power of two: the row's values are its codes
 *                     times its scale
 * head_dim is 64 or 128, page_size a multiple of 16. */
typedef struct gemm_epi_paged_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t num_pages;
  int64_t page_size;
  int64_t heads;
  int64_t head_dim;
  gemm_epi_dtype dtype;
} gemm_epi_paged_cache;

/* The sequences of a call: token p of sequence i is in slot p % page_size of
 * page pages[i * ld + p / page_size], and the sequence holds lens[i] tokens,
 * those appended by the current step included.  Both arrays are in device
 * memory and are read when the kernel runs, so a captured graph follows
 * what they hold at its replay.
 * An entry outside [0, num_pages) is no page: nothing is written there, and
 * its tokens take no part in the attention.  A length is taken as clamped
 * to [0, width * page_size]. */
typedef struct gemm_epi_page_table {
  const int32_t* pages; /* [batch, ld] */
  int64_t ld;           /* elements between the rows of `pages`, at least width */
  int64_t width;        /* pages a sequence can have */
  const int32_t* lens;  /* [batch] */
  int64_t batch;
} gemm_epi_page_table;

/* gemm_epi_cache_append -- write the keys and values of new tokens into the
 * cache.
 *
 *   K, V    [tokens, heads, head_dim], format `dtype` (F16 or BF16), ldk and
 *           ldv elements between tokens (the heads of a token contiguous), so
 *           that both can be columns of one projection's output
 *   starts  batch + 1 ascending token numbers: the rows of sequence i are
 *           [starts[i], starts[i + 1]); rows from starts[batch] on belong to
 *           no sequence and are ignored.  NULL: one row a sequence (tokens =
 *           batch).
 * The new tokens of sequence i are its last ones: row t goes to position
 * lens[i] - (starts[i + 1] - t); a position below 0 or at or past width *
 * page_size is not written.
 * The cache has the format of K and V (the rows are copied), or FP8_E4M3:
 * scale 2^e with e the smallest integer, -100 at least, such that max|x| <=
 * 448 * 2^e over the row's head_dim values, and codes x / 2^e rounded to
 * nearest even; a row that holds an infinity or a NaN gets scale NaN (all its
 * values read as NaN).
 * No two rows may fall on the same slot of the cache (two sequences that
 * share the page they append to): which one stays is then not defined.
 * tokens = 0 or batch = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer, a negative or zero size, an ld below
 * its minimum, tokens != batch without starts, the formats do not fit),
 * UNSUPPORTED (head_dim not 64 or 128, page_size not a multiple of 16 or
 * above 65536, more than 1024 heads, num_pages * page_size >= 2^31, width *
 * page_size above 2^31 - 256, batch times the 128-token units of width *
 * page_size >= 2^31, tokens above 2^26 - 4, batch > 65535; a pointer of the cache, K
 * or V that is not 16-byte aligned, ldk or ldv not a multiple of 8), HIP. */
gemm_epi_status gemm_epi_cache_append(const gemm_epi_paged_cache* cache, const gemm_epi_page_table* table,
                                      const void* K, int64_t ldk, const void* V, int64_t ldv, const int32_t* starts,
                                      int64_t tokens, gemm_epi_dtype dtype, void* stream);

#define GEMM_EPI_ATTENTION_DECODE_COUNTER_BYTES 2048

/* gemm_epi_attention_decode -- attention of one new token of each sequence
 * over its cache,
 *
 *     O[i, h] = sum_j softmax_j(Q[i, h] . K_j / sqrt(head_dim)) V_j
 *
 * over the tokens j < lens[i] of sequence i whose page exists, with K_j and
 * V_j of key head h / (q_heads / heads).  No such token, or only minus infinities
 * for scores: O[i, h] = 0.
 *   Q   [batch, q_heads, head_dim], ldq elements between sequences, format
 *       `dtype` (F16 or BF16), that of the cache unless that is FP8_E4M3
 *   O   [batch, q_heads, head_dim], ldo elements between sequences, `dtype`
 * O overlaps nothing else.  q_heads is a multiple of the cache's heads.  What
 * the cache holds at or past a sequence's length, in pages of no sequence or
 * in the scales there is read into no result, NaN included.
 * Scores, softmax and accumulation in fp32; the probabilities enter the
 * second product as two 16-bit parts (their rounded value and its rounded
 * remainder), in F16 of 2^7 times their ratio to the largest, in BF16 and for
 * an FP8_E4M3 cache in BF16; such a cache's values enter both products exactly
 * (from 2^128 on as infinities); O is rounded once.  What attends to an
 * infinity of V is an infinity or NaN.  The keys are split over workgroups by
 * the lengths found on the device and joined in a fixed order: the same inputs
 * give the same bits.
 * workspace: gemm_epi_attention_decode_workspace_size bytes, 16-byte aligned.
 * Its first GEMM_EPI_ATTENTION_DECODE_COUNTER_BYTES hold counters: zero-filled
 * once before its first use, and left zero by every run that completes; the
 * rest has no content of its own before or after a call.  One workspace
 * serves calls of any sizes it is large enough for; runs that share it must
 * not overlap in time.
 * batch = 0 does nothing.
 * Errors: INVALID_ARG (a NULL pointer, a negative or zero size, q_heads not a
 * multiple of the cache's heads, an ld below its minimum, formats that do
 * not fit, workspace missing or too small),
 * UNSUPPORTED (the cache's and table's limits of gemm_epi_cache_append; Q, O
 * or workspace not 16-byte aligned, ldq or ldo not a multiple of 8, more than
 * 16384 query heads, batch times the 128-token units of width * page_size
 * times heads times the tiles of 16 query heads of a key head >= 2^31), HIP. */
gemm_epi_status gemm_epi_attention_decode(const gemm_epi_paged_cache* cache, const gemm_epi_page_table* table,
                                          const void* Q, int64_t ldq, void* O, int64_t ldo, int64_t q_heads,
                                          gemm_epi_dtype dtype, void* workspace, size_t workspace_bytes,
                                          void* stream);

/* Bytes of workspace for batches of up to `batch` sequences of up to `width`
 * pages (0 for sizes that the call would refuse).  Host only; of the cache
 * only its sizes are read. */
size_t gemm_epi_attention_decode_workspace_size(const gemm_epi_paged_cache* cache, int64_t batch, int64_t width,
                                                int64_t q_heads);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPI_DECODE_H */
