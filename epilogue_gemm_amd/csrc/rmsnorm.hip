// rmsnorm.hip -- root-mean-square norm with the residual's addition:
//
//     h = x + r        y = h / sqrt(mean(h^2) + eps) * w
//
// per row, in fp32; h and y rounded once, y optionally to E4M3 with the
// row's scale max|y| / 448.  HBM-bound for many rows (x and r read, h and y
// written, once each), bound by one launch and one reduction's latency for
// few (16384 x 8192 bf16 with a residual 178 us, 6.0 TB/s; 8191 x 5120 f16 to
// E4M3 26.7 us; 4 x 4096 2.7 us).  Storing past the caches was faster alone and
// not kept, as the reader that follows pays for it (8192 x 5120 to E4M3 26.6
// against 23.0 us, with a reading of y 33.4 against 34.6).
#include "kernels.hpp"
#include "rows.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_decode.h"

namespace ge {
namespace norm {

using rows::load8;
using rows::store8;
using rows::widen;

struct Args {
  const void *X, *R, *W;
  void *H, *Y;
  float* y_scale;
  int64_t ldx, ldr, ldh, ldy;
  int rows, cols;
  float eps;
};

// A row in the registers of a workgroup's waves (LPR = 0), or of LPR = 16
// lanes of one of four waves, each lane VPT pieces of eight values: every
// tensor is read or written once, each place by one thread, which has read
// what H or Y may overwrite there before it writes.  All loads, the weights'
// included, are issued before anything waits, and the sum and an E4M3
// output's largest |h w| (its scale needs only that times 1 / rms) cross the
// waves together: one memory latency and one barrier a row.
template <typename T, typename TOut, bool ANY, int VPT, int LPR>
__global__ __launch_bounds__(LPR ? 256 : 1024) void rmsnorm_rows(Args a) {
  constexpr bool FP8 = sizeof(TOut) == 1;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  __shared__ f32x2 part[2][16];  // of alternate rows
  constexpr int RPB = LPR ? 256 / LPR : 1;  // rows a workgroup
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int at = (LPR ? threadIdx.x % LPR : threadIdx.x) * 8, step = (LPR ? LPR : (int)blockDim.x) * 8;
  const int64_t row0 = (int64_t)blockIdx.x * RPB + (LPR ? threadIdx.x / LPR : 0);
  int slot = 0;
  for (int64_t row = row0; row < a.rows; row += (int64_t)gridDim.x * RPB, slot ^= 1) {
    const uint16_t* x = (const uint16_t*)a.X + row * a.ldx;
    const uint16_t* r = a.R ? (const uint16_t*)a.R + row * a.ldr : nullptr;
    u32x4 xr[VPT], rr[VPT], wr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) xr[i] = load8<ANY>(x, at + i * step, a.cols);
    if (r) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) rr[i] = load8<ANY>(r, at + i * step, a.cols);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) wr[i] = load8<ANY>((const uint16_t*)a.W, at + i * step, a.cols);
    float h[VPT][8];  // h, then h w
    float ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
      widen<T>(xr[i], h[i]);
      if (r) {
        widen<T>(rr[i], f);
#pragma unroll
        for (int u = 0; u < 8; ++u) h[i][u] += f[u];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) ss = __builtin_fmaf(h[i][u], h[i][u], ss);
      if (a.H) store8<T, ANY>((T*)a.H + row * a.ldh, at + i * step, a.cols, h[i]);
      widen<T>(wr[i], f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        h[i][u] *= f[u];
        if constexpr (FP8) mx = fmaxf(mx, fabsf(h[i][u]));
      }
    }
    ss = LPR == 16 ? wave::over_row<wave::Sum>(ss) : wave::all<wave::Sum>(ss);
    if constexpr (FP8) mx = LPR == 16 ? wave::over_row<wave::Max>(mx) : wave::all<wave::Max>(mx);
    if constexpr (LPR == 0) {
      // (a wave that is a row ahead writes the other slot, and none can be
      // two ahead of a wave still reading)
      if ((threadIdx.x & 63) == 0) part[slot][wave] = f32x2{ss, mx};
      __syncthreads();
      ss = 0.0f;
      for (int i = 0; i < waves; ++i) {
        ss += part[slot][i].x;
        if constexpr (FP8) mx = fmaxf(mx, part[slot][i].y);
      }
    }
    const float rs = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    float inv = 1.0f;  // (apart from rs: their product may overflow, for a tiny eps)
    if constexpr (FP8) {
      const float s = fmaxf(mx * rs / 448.0f, 0x1p-100f);
      inv = 1.0f / s;
      if (at == 0) a.y_scale[row] = s;
    }
    TOut* yp = (TOut*)a.Y + row * a.ldy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int u = 0; u < 8; ++u) h[i][u] = FP8 ? h[i][u] * rs * inv : h[i][u] * rs;
      store8<TOut, ANY>(yp, at + i * step, a.cols, h[i]);
    }
  }
}

// Rows longer than a workgroup's registers: one workgroup a row, read once
// for the sum, once more for the largest |y| of an E4M3 output, and once for
// the outputs (each element is read by the thread that then writes its
// place, so that H and Y may be X or R).
template <typename T, typename TOut>
__global__ __launch_bounds__(1024) void rmsnorm_long(Args a) {
  __shared__ float part[2][16];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.X + row * a.ldx;
    const T* r = a.R ? (const T*)a.R + row * a.ldr : nullptr;
    const T* w = (const T*)a.W;
    T* hp = a.H ? (T*)a.H + row * a.ldh : nullptr;
    TOut* yp = (TOut*)a.Y + row * a.ldy;
    auto load = [&](int64_t j) { return to_f32(x[j]) + (r ? to_f32(r[j]) : 0.0f); };
    float ss = 0.0f;
    for (int64_t j = tid; j < a.cols; j += 1024) {
      const float h = load(j);
      ss = __builtin_fmaf(h, h, ss);
    }
    ss = wave::all<wave::Sum>(ss);
    if ((tid & 63) == 0) part[0][tid >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < 16; ++i) ss += part[0][i];
    const float rs = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    float inv = 1.0f;
    if constexpr (sizeof(TOut) == 1) {
      float mx = 0.0f;
      for (int64_t j = tid; j < a.cols; j += 1024) mx = fmaxf(mx, fabsf(load(j) * rs * to_f32(w[j])));
      mx = wave::all<wave::Max>(mx);
      if ((tid & 63) == 0) part[1][tid >> 6] = mx;
      __syncthreads();
      mx = 0.0f;
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, part[1][i]);
      const float s = fmaxf(mx / 448.0f, 0x1p-100f);
      inv = 1.0f / s;
      if (tid == 0) a.y_scale[row] = s;
    }
    for (int64_t j = tid; j < a.cols; j += 1024) {
      const float h = load(j);
      float y = h * rs * to_f32(w[j]);
      if constexpr (sizeof(TOut) == 1) y *= inv;
      if (hp) hp[j] = from_f32<T>(h);
      yp[j] = from_f32<TOut>(y);
    }
    __syncthreads();  // `part` is free for the next row
  }
}

constexpr int kMaxGrid = 1 << 20;  // a grid's threads fit 32 bits; further rows by the kernels' loops

template <typename T, typename TOut, bool ANY, int VPT, int LPR>
hipError_t launch_rows(const Args& a, hipStream_t stream) {
  constexpr int RPB = LPR ? 256 / (LPR + !LPR) : 1;
  const int wgs = (int)(((int64_t)a.rows + RPB - 1) / RPB);
  const int waves = LPR ? 4 : (a.cols + 512 * VPT - 1) / (512 * VPT);
  hipLaunchKernelGGL((rmsnorm_rows<T, TOut, ANY, VPT, LPR>), dim3(min(wgs, kMaxGrid)), dim3(64 * waves), 0, stream, a);
  return hipGetLastError();
}

// Pieces per lane.  One, with as many waves as that takes, gives a row the
// shortest latency (4 rows of 4096 with a residual: 2.5 us, two pieces 3.0)
// and is as fast for many where a residual doubles the bytes in flight
// (16384 x 8192 bf16: 181 against 188 us).  Many rows without one want two
// (8192 x 8192 f16 to E4M3: 44 against 54 us; 8192 x 8192 bf16: 54 against
// 61).  Longer rows take what their 16 waves need.  Up to 128 columns a row
// is 16 lanes' (200000 x 128: 38 us, a wave each 57).
template <typename T, typename TOut, bool ANY>
hipError_t launch_any(const Args& a, hipStream_t stream) {
  if (a.cols <= 128) return launch_rows<T, TOut, ANY, 1, 16>(a, stream);
  if (a.cols <= 512 || (a.cols <= 8192 && (a.R || a.rows < 1024))) return launch_rows<T, TOut, ANY, 1, 0>(a, stream);
  if (a.cols <= 16384) return launch_rows<T, TOut, ANY, 2, 0>(a, stream);
  if (a.cols <= 32768) return launch_rows<T, TOut, ANY, 4, 0>(a, stream);
  hipLaunchKernelGGL((rmsnorm_long<T, TOut>), dim3(min(a.rows, kMaxGrid)), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

template <typename T, typename TOut>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int64_t lds = a.cols | a.ldx | a.ldy | (a.R ? a.ldr : 0) | (a.H ? a.ldh : 0);
  const uintptr_t ptrs = (uintptr_t)a.X | (uintptr_t)a.R | (uintptr_t)a.W | (uintptr_t)a.H |
                         (sizeof(TOut) == 1 ? (uintptr_t)a.Y << 1 : (uintptr_t)a.Y);
  const bool aligned = (lds & 7) == 0 && (ptrs & 15u) == 0;
  return aligned ? launch_any<T, TOut, false>(a, stream) : launch_any<T, TOut, true>(a, stream);
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
  if (rows < 0 || cols <= 0 || !(eps >= 0.0f) || eps == __builtin_inff()) return GEMM_EPI_ERR_INVALID_ARG;
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
