// grouped.cpp -- the entries of the products grouped by expert and of the
// product of 8-bit integers: their argument checks.
#include "grouped.hpp"

namespace ge {
namespace grouped {
namespace {

constexpr int64_t kLim = (int64_t)1 << 31;

gemm_epi_status status_of(hipError_t e) {
  if (e == hipSuccess) return GEMM_EPI_OK;
  set_last_hip_error((int)e);
  return GEMM_EPI_ERR_HIP;
}

bool half(gemm_epi_dtype t) { return t == GEMM_EPI_F16 || t == GEMM_EPI_BF16; }
bool known(gemm_epi_epilogue e) { return (int)e >= GEMM_EPI_NONE && (int)e <= GEMM_EPI_BIAS_SILU; }
bool biased(gemm_epi_epilogue e) {
  return e == GEMM_EPI_BIAS || e == GEMM_EPI_BIAS_RELU || e == GEMM_EPI_BIAS_GELU || e == GEMM_EPI_BIAS_SILU;
}

// Blocks of 16 x 16 outputs, of which no kernel takes fewer than one for 64
// threads: a grid holds below 2^32.
bool too_many(int64_t rows, int64_t groups, int64_t cols) {
  return ((rows + 15) / 16 + std::min(groups, rows)) * ((cols + 15) / 16) > ((int64_t)1 << 25);
}

// Bytes between rows: a tile's rows are at 32-bit offsets from its first.
constexpr int64_t kMaxPitch = (int64_t)1 << 24;
// Bytes of a group's gates: the values' rows are at 32-bit offsets from them.
constexpr int64_t kMaxGate = (int64_t)1 << 31;

}  // namespace
}  // namespace grouped
}  // namespace ge

extern "C" {

gemm_epi_status gemm_epi_i8_gemm(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                                 const float* b_scale, const void* bias, const void* R, int64_t ldr, void* C,
                                 int64_t ldc, int64_t M, int64_t N, int64_t K, gemm_epi_epilogue epilogue,
                                 gemm_epi_dtype out_dtype, void* stream) {
  using namespace ge::grouped;
  if (!half(out_dtype) || !known(epilogue) || M < 0 || N <= 0 || K <= 0 || lda < K || ldb < K || ldc < N ||
      (R && ldr < N))
    return GEMM_EPI_ERR_INVALID_ARG;
  if ((((uintptr_t)a_scale | (uintptr_t)b_scale) & 3u) || (((uintptr_t)R | (uintptr_t)C) & 1u) ||
      (biased(epilogue) && ((uintptr_t)bias & 1u)))
    return GEMM_EPI_ERR_INVALID_ARG;
  for (const int64_t n : {M, N, ldc, R ? ldr : 0})
    if (n >= kLim) return GEMM_EPI_ERR_UNSUPPORTED;
  if (K % 16 != 0 || K >= (1 << 17) || lda % 16 != 0 || ldb % 16 != 0 || lda > kMaxPitch || ldb > kMaxPitch ||
      too_many(M, 1, N))
    return GEMM_EPI_ERR_UNSUPPORTED;
  if (M == 0) return GEMM_EPI_OK;
  if (!A || !B || !C || !a_scale || !b_scale || (biased(epilogue) && !bias)) return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)A | (uintptr_t)B) & 15u) return GEMM_EPI_ERR_UNSUPPORTED;
  Args a{};
  a.X = A, a.W = B, a.bias = bias, a.R = R, a.xs = a_scale, a.ws = b_scale, a.C = C;
  a.ldx = lda, a.ldw = ldb, a.ldr = ldr, a.ldc = ldc;
  a.groups = 1, a.rows = (int)M, a.per = 1, a.N = (int)N, a.K = (int)K;
  a.epi = (int)epilogue;
  const hipStream_t s = (hipStream_t)stream;
  return status_of(out_dtype == GEMM_EPI_F16 ? launch_i8_f16(a, false, s) : launch_i8_bf16(a, false, s));
}

gemm_epi_status gemm_epi_grouped_gemm(const gemm_epi_groups* groups, const void* X, int64_t ldx, const float* x_scale,
                                      const void* W, const float* w_scale, const void* bias, void* C, int64_t ldc,
                                      int64_t N, int64_t K, int flags, gemm_epi_epilogue epilogue,
                                      gemm_epi_dtype dtype, gemm_epi_dtype out_dtype, void* stream) {
  using namespace ge::grouped;
  const bool i8 = dtype == GEMM_EPI_I8;
  if (!groups || (!i8 && !half(dtype)) || (i8 ? !half(out_dtype) : out_dtype != dtype) || !known(epilogue) ||
      (flags & ~(GEMM_EPI_GATHER | GEMM_EPI_SCATTER | GEMM_EPI_GATED)))
    return GEMM_EPI_ERR_INVALID_ARG;
  const gemm_epi_groups& g = *groups;
  const bool gather = flags & GEMM_EPI_GATHER, scatter = flags & GEMM_EPI_SCATTER, gated = flags & GEMM_EPI_GATED;
  if (g.rows < 0 || g.groups <= 0 || g.per <= 0 || N <= 0 || K <= 0 || ldx < K || ldc < N ||
      (gather && g.rows % g.per != 0))
    return GEMM_EPI_ERR_INVALID_ARG;
  if ((((uintptr_t)g.offsets | (uintptr_t)g.order | (uintptr_t)x_scale | (uintptr_t)w_scale) & 3u) ||
      ((uintptr_t)C & 1u) || (biased(epilogue) && ((uintptr_t)bias & 1u)))
    return GEMM_EPI_ERR_INVALID_ARG;
  // (each bounded by itself before a product of it is formed)
  for (const int64_t n : {g.rows, g.per, N, ldx, ldc})
    if (n >= kLim) return GEMM_EPI_ERR_UNSUPPORTED;
  if (K >= (1 << 17) || g.groups > 1024) return GEMM_EPI_ERR_UNSUPPORTED;
  const int64_t size = i8 ? 1 : 2, cols = gated ? 2 * N : N, pitch = ldx * size;
  if ((gated && N * K * size > kMaxGate) || K * size % 16 != 0 || pitch % 16 != 0 || pitch > kMaxPitch || cols >= kLim ||
      too_many(g.rows, g.groups, cols) || (gather && g.rows / g.per * pitch >= (int64_t)0xffff0000))
    return GEMM_EPI_ERR_UNSUPPORTED;
  if (g.rows == 0) return GEMM_EPI_OK;
  if (!g.offsets || ((gather || scatter) && !g.order) || !X || !W || !C || i8 != (x_scale != nullptr) ||
      i8 != (w_scale != nullptr) || (biased(epilogue) && !bias))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)X | (uintptr_t)W) & 15u) return GEMM_EPI_ERR_UNSUPPORTED;
  Args a{};
  a.offsets = g.offsets, a.order = g.order;
  a.X = X, a.W = W, a.bias = bias, a.xs = x_scale, a.ws = w_scale, a.C = C;
  a.ldx = ldx, a.ldw = K, a.ldc = ldc, a.group_w = cols * K;
  a.groups = (int)g.groups, a.rows = (int)g.rows, a.per = (int)g.per, a.N = (int)N, a.K = (int)K;
  a.gather = gather, a.scatter = scatter, a.epi = (int)epilogue;
  const hipStream_t s = (hipStream_t)stream;
  if (i8) return status_of(out_dtype == GEMM_EPI_F16 ? launch_i8_f16(a, gated, s) : launch_i8_bf16(a, gated, s));
  return status_of(dtype == GEMM_EPI_F16 ? launch_f16_f16(a, gated, s) : launch_bf16_bf16(a, gated, s));
}

}  // extern "C"
