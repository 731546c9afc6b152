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

// V consecutive values (8, or 1 where rows are not 16-byte aligned) as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float (&f)[V]) {
  if constexpr (V == 8) {
    const u32x4 w = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = to_f32(__builtin_bit_cast(T, (uint16_t)(w[i] & 0xffffu)));
      f[2 * i + 1] = to_f32(__builtin_bit_cast(T, (uint16_t)(w[i] >> 16)));
    }
  } else {
    f[0] = to_f32(p[0]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    p[0] = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 1) {
    *(u32x2*)p = u32x2{pack4_e4m3(f[0], f[1], f[2], f[3]), pack4_e4m3(f[4], f[5], f[6], f[7])};
  } else {
    *(u32x4*)p = u32x4{pack2_out<T>(f[0], f[1]), pack2_out<T>(f[2], f[3]), pack2_out<T>(f[4], f[5]),
                       pack2_out<T>(f[6], f[7])};
  }
}

// A row in the registers of WPR waves (1 or 4: 256 threads, 4 or 1 rows a
// workgroup; 16: 1024 threads), each lane VPT pieces of V values: every
// tensor is read or written once, and H or Y may be X or R, since a row is
// whole in registers before the reduction that precedes its first store.
template <typename T, typename TOut, int V, int WPR, int VPT>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 256) void rmsnorm_rows(Args a) {
  constexpr int RPB = WPR == 1 ? 4 : 1;
  __shared__ float part[2][WPR];
  const int wave = threadIdx.x >> 6;
  const int at = (WPR == 1 ? (threadIdx.x & 63) : threadIdx.x) * V;
  constexpr int step = WPR * 64 * V;
  auto reduce = [&](float v, int slot, bool max_of) {
    v = max_of ? wave_max(v) : wave_sum(v);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 63) == 0) part[slot][wave] = v;
      __syncthreads();
      v = part[slot][0];
#pragma unroll
      for (int i = 1; i < WPR; ++i) v = max_of ? fmaxf(v, part[slot][i]) : v + part[slot][i];
    }
    return v;
  };
  for (int64_t row = (int64_t)blockIdx.x * RPB + (WPR == 1 ? wave : 0); row < a.rows; row += (int64_t)gridDim.x * RPB) {
    const T* x = (const T*)a.X + row * a.ldx;
    float h[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int j = at + i * step;
#pragma unroll
      for (int u = 0; u < V; ++u) h[i][u] = 0.0f;
      if (j < a.cols) load_row<T, V>(x + j, h[i]);
    }
    if (a.R) {
      const T* r = (const T*)a.R + row * a.ldr;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int j = at + i * step;
        float f[V] = {};
        if (j < a.cols) load_row<T, V>(r + j, f);
#pragma unroll
        for (int u = 0; u < V; ++u) h[i][u] += f[u];
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u) ss = __builtin_fmaf(h[i][u], h[i][u], ss);
    ss = reduce(ss, 0, false);
    const float rs = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    if (a.H) {
      T* hp = (T*)a.H + row * a.ldh;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (at + i * step < a.cols) store_row<T, V>(hp + at + i * step, h[i]);
    }
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int j = at + i * step;
      float w[V] = {};
      if (j < a.cols) load_row<T, V>((const T*)a.W + j, w);
#pragma unroll
      for (int u = 0; u < V; ++u) {
        h[i][u] = h[i][u] * rs * w[u];
        if (sizeof(TOut) == 1) mx = fmaxf(mx, fabsf(h[i][u]));
      }
    }
    if constexpr (sizeof(TOut) == 1) {
      const float s = fmaxf(reduce(mx, 1, true) / 448.0f, 0x1p-100f), inv = 1.0f / s;
      if (at == 0) a.y_scale[row] = s;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int u = 0; u < V; ++u) h[i][u] *= inv;
    }
    TOut* yp = (TOut*)a.Y + row * a.ldy;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (at + i * step < a.cols) store_row<TOut, V>(yp + at + i * step, h[i]);
    if constexpr (WPR > 1) __syncthreads();  // `part` is free for the next row
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
    ss = wave_sum(ss);
    if ((tid & 63) == 0) part[0][tid >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < 16; ++i) ss += part[0][i];
    const float rs = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    float inv = 1.0f;
    if constexpr (sizeof(TOut) == 1) {
      float mx = 0.0f;
      for (int64_t j = tid; j < a.cols; j += 1024) mx = fmaxf(mx, fabsf(load(j) * rs * to_f32(w[j])));
      mx = wave_max(mx);
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

template <typename T, typename TOut, int V, int WPR, int VPT>
hipError_t launch_rows(const Args& a, hipStream_t stream) {
  const int wgs = WPR == 1 ? (a.rows + 3) / 4 : a.rows;
  hipLaunchKernelGGL((rmsnorm_rows<T, TOut, V, WPR, VPT>), dim3(min(wgs, kMaxGrid)), dim3(WPR == 16 ? 1024 : 256), 0,
                     stream, a);
  return hipGetLastError();
}

// The fewest waves whose registers hold a row: 8-value pieces where every
// row of every tensor allows 16-byte accesses, else single values.
template <typename T, typename TOut>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int64_t lds = a.ldx | a.ldy | (a.R ? a.ldr : 0) | (a.H ? a.ldh : 0);
  const uintptr_t ptrs = (uintptr_t)a.X | (uintptr_t)a.R | (uintptr_t)a.W | (uintptr_t)a.H |
                         (sizeof(TOut) == 1 ? (uintptr_t)a.Y << 1 : (uintptr_t)a.Y);
  if (a.cols % 8 == 0 && (lds & 7) == 0 && (ptrs & 15u) == 0) {
    if (a.cols <= 512) return launch_rows<T, TOut, 8, 1, 1>(a, stream);
    if (a.cols <= 2048) return launch_rows<T, TOut, 8, 4, 1>(a, stream);
    if (a.cols <= 4096) return launch_rows<T, TOut, 8, 4, 2>(a, stream);
    if (a.cols <= 8192) return launch_rows<T, TOut, 8, 4, 4>(a, stream);
    if (a.cols <= 16384) return launch_rows<T, TOut, 8, 16, 2>(a, stream);
    if (a.cols <= 32768) return launch_rows<T, TOut, 8, 16, 4>(a, stream);
  } else {
    if (a.cols <= 256) return launch_rows<T, TOut, 1, 1, 4>(a, stream);
    if (a.cols <= 1024) return launch_rows<T, TOut, 1, 4, 4>(a, stream);
    if (a.cols <= 4096) return launch_rows<T, TOut, 1, 4, 16>(a, stream);
    if (a.cols <= 16384) return launch_rows<T, TOut, 1, 16, 16>(a, stream);
  }
  hipLaunchKernelGGL((rmsnorm_long<T, TOut>), dim3(min(a.rows, kMaxGrid)), dim3(1024), 0, stream, a);
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
