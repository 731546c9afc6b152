// rmsnorm.hip -- root-mean-square norm with the residual's addition:
//
//     h = x + r        y = h / sqrt(mean(h^2) + eps) * w
//
// per row, in fp32; h and y rounded once, y optionally to E4M3 with the
// row's scale max|y| / 448.  HBM-bound for many rows (x and r read, h and y
// written, once each), bound by one launch and one reduction's latency for
// few.
#include "common.hpp"
#include "kernels.hpp"

#include "../../include/gemm_epi_decode.h"

namespace ge {
namespace norm {

struct Args {
  const void *X, *R, *W;
  void *H, *Y;
  float* y_scale;
  int64_t ldx, ldr, ldh, ldy;
  int rows, cols;
  float eps;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Any column count, alignment and leading dimension: one workgroup a row,
// the row read once for the sum, once more for the largest |y| of an E4M3
// output, and once for the outputs (each element is read by the thread that
// then writes its place, so that H and Y may be X or R).
template <typename T, typename TOut>
__global__ __launch_bounds__(256) void rmsnorm_any(Args a) {
  __shared__ float part[2][4];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
  const T* x = (const T*)a.X + row * a.ldx;
  const T* r = a.R ? (const T*)a.R + row * a.ldr : nullptr;
  const T* w = (const T*)a.W;
  T* hp = a.H ? (T*)a.H + row * a.ldh : nullptr;
  TOut* yp = (TOut*)a.Y + row * a.ldy;
  auto load = [&](int j) { return to_f32(x[j]) + (r ? to_f32(r[j]) : 0.0f); };
  float ss = 0.0f;
  for (int j = tid; j < a.cols; j += 256) {
    const float h = load(j);
    ss = __builtin_fmaf(h, h, ss);
  }
  ss = wave_sum(ss);
  if ((tid & 63) == 0) part[0][tid >> 6] = ss;
  __syncthreads();
  ss = part[0][0] + part[0][1] + part[0][2] + part[0][3];
  const float rs = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
  float inv = 1.0f;
  if constexpr (sizeof(TOut) == 1) {
    float mx = 0.0f;
    for (int j = tid; j < a.cols; j += 256) mx = fmaxf(mx, fabsf(load(j) * rs * to_f32(w[j])));
    mx = wave_max(mx);
    if ((tid & 63) == 0) part[1][tid >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(part[1][0], part[1][1]), fmaxf(part[1][2], part[1][3]));
    const float s = fmaxf(mx / 448.0f, 0x1p-100f);
    inv = 1.0f / s;
    if (tid == 0) a.y_scale[row] = s;
  }
  for (int j = tid; j < a.cols; j += 256) {
    const float h = load(j);
    float y = h * rs * to_f32(w[j]);
    if constexpr (sizeof(TOut) == 1) y *= inv;
    if (hp) hp[j] = from_f32<T>(h);
    yp[j] = from_f32<TOut>(y);
  }
  __syncthreads();  // `part` is free for the next row
  }
}

template <typename T, typename TOut>
hipError_t launch(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((rmsnorm_any<T, TOut>), dim3(min(a.rows, 1 << 20)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace norm
}  // namespace ge

extern "C" gemm_epi_status gemm_epi_rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* W,
                                            void* H, int64_t ldh, void* Y, int64_t ldy, float* y_scale, int64_t rows,
                                            int64_t cols, float eps, gemm_epi_dtype dtype, gemm_epi_dtype out_dtype,
                                            void* stream) {
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_INVALID_ARG;
  const bool fp8 = out_dtype == GEMM_EPI_FP8_E4M3;
  if (!fp8 && out_dtype != dtype) return GEMM_EPI_ERR_INVALID_ARG;
  if (rows < 0 || cols <= 0 || !(eps >= 0.0f) || eps > 3.0e38f) return GEMM_EPI_ERR_INVALID_ARG;
  if (ldx < cols || ldy < cols || (R && ldr < cols) || (H && ldh < cols)) return GEMM_EPI_ERR_INVALID_ARG;
  if (!X || !W || !Y || fp8 != (y_scale != nullptr)) return GEMM_EPI_ERR_INVALID_ARG;
  const int64_t lim = (int64_t)1 << 31;
  if (rows >= lim || cols >= lim) return GEMM_EPI_ERR_UNSUPPORTED;
  for (const void* p : {X, R, W, (const void*)H, fp8 ? (const void*)nullptr : (const void*)Y})
    if ((uintptr_t)p & 1u) return GEMM_EPI_ERR_INVALID_ARG;
  if ((uintptr_t)y_scale & 3u) return GEMM_EPI_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_EPI_OK;
  const ge::norm::Args a{X, R, W, H, Y, y_scale, ldx, ldr, ldh, ldy, (int)rows, (int)cols, eps};
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      dtype == GEMM_EPI_F16
          ? (fp8 ? ge::norm::launch<ge::f16, ge::fp8e4m3>(a, s) : ge::norm::launch<ge::f16, ge::f16>(a, s))
          : (fp8 ? ge::norm::launch<ge::bf16, ge::fp8e4m3>(a, s) : ge::norm::launch<ge::bf16, ge::bf16>(a, s));
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}
