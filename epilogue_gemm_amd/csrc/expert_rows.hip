// expert_rows.hip -- passes over rows beside the experts' products: rows in
// 8-bit integers,
//
//     scale = max(max|x| / 127, 2^-100)        y = rint(x / scale)
//
// and a token's rows brought together,
//
//     y = r + sum_j w_j z_j
//
// each tensor read or written once.  Bound by HBM for many rows, by a launch
// and a memory latency for few.
#include <algorithm>

#include "kernels.hpp"
#include "rows.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_experts.h"

namespace ge {
namespace rows {

// ---------------------------------------------------------------------------
// rows in 8-bit integers
// ---------------------------------------------------------------------------
struct QuantArgs {
  const void* X;
  int8_t* Y;
  float* scale;
  int64_t ldx, ldy;
  int rows, cols;
};

// The larger of two values >= 0 by their bits, which order a NaN above every
// number.
struct MaxBits {
  __device__ static __forceinline__ float op(float a, float b) {
    return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)));
  }
};

template <typename T>
__device__ __forceinline__ float largest(u32x4 w, float mx) {
  float f[8];
  widen<T>(w, f);
#pragma unroll
  for (int u = 0; u < 8; ++u) mx = MaxBits::op(mx, __builtin_fabsf(f[u]));
  return mx;
}

// The scale of a row whose largest value is mx.
__device__ __forceinline__ float scale_of(float mx) {
  return mx < __builtin_inff() ? fmaxf(mx / 127.0f, 0x1p-100f) : __builtin_nanf("");
}

// Eight quotients as bytes; a scale of NaN: zeros.  The product with the scale's
// reciprocal is within 128 * 3 * 2^-24 of the quotient, so that it rounds to the
// same integer unless it lies within 2^-14 of the middle between two: the
// quotients themselves are formed where one of a wave's does (eight divisions a
// lane always: 57 us for 16383 x 5120).
template <typename T, bool ANY>
__device__ __forceinline__ void quantise8(int8_t* row, int j, int cols, u32x4 x, float s, float inv) {
  if (j >= cols) return;
  float f[8], q[8], near = 1.0f;
  widen<T>(x, f);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float p = f[u] * inv;
    q[u] = __builtin_rintf(p);
    near = fminf(near, 0.5f - __builtin_fabsf(p - q[u]));
  }
  if (near < 0x1p-14f) {
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u] = __builtin_rintf(f[u] / s);
  }
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // (whole numbers of at most 128: in the lowest byte as integers)
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)(int)q[4 * i + 1], (uint32_t)(int)q[4 * i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)(int)q[4 * i + 3], (uint32_t)(int)q[4 * i + 2], 0x04000c0cu);
    w[i] = s == s ? lo | hi : 0u;
  }
  if (ANY && j + 8 > cols) {
    for (int u = 0; u < 8; ++u)
      if (j + u < cols) row[j + u] = (int8_t)(w[u >> 2] >> (8 * (u & 3)));
    return;
  }
  if constexpr (ANY) *(u32x2_any*)(row + j) = w;
  else *(u32x2*)(row + j) = w;
}

// A row in the registers of a workgroup's waves (LPR = 0), or of LPR = 16
// lanes of one of four waves, each lane VPT pieces of eight values.
template <typename T, bool ANY, int VPT, int LPR, bool PAST>
__global__ __launch_bounds__(LPR ? 256 : 1024) void quantise_rows(QuantArgs a) {
  __shared__ float part[2][16];  // of alternate rows
  constexpr int RPB = LPR ? 256 / LPR : 1;
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int at = (LPR ? threadIdx.x % LPR : threadIdx.x) * 8, step = (LPR ? LPR : (int)blockDim.x) * 8;
  const int64_t row0 = (int64_t)blockIdx.x * RPB + (LPR ? threadIdx.x / LPR : 0);
  int slot = 0;
  for (int64_t row = row0; row < a.rows; row += (int64_t)gridDim.x * RPB, slot ^= 1) {
    const uint16_t* x = (const uint16_t*)a.X + row * a.ldx;
    u32x4 xr[VPT];
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) xr[i] = load8<ANY, PAST>(x, at + i * step, a.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) mx = largest<T>(xr[i], mx);
    mx = LPR == 16 ? wave::over_row<MaxBits>(mx) : wave::all<MaxBits>(mx);
    if constexpr (LPR == 0) {
      // (a wave that is a row ahead writes the other slot, and none can be
      // two ahead of a wave still reading)
      if ((threadIdx.x & 63) == 0) part[slot][wave] = mx;
      __syncthreads();
      for (int i = 0; i < waves; ++i) mx = MaxBits::op(mx, part[slot][i]);
    }
    const float s = scale_of(mx);
    const float inv = 1.0f / s;
    if (at == 0) a.scale[row] = s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) quantise8<T, ANY>(a.Y + row * a.ldy, at + i * step, a.cols, xr[i], s, inv);
  }
}

// Rows longer than a workgroup's registers: read twice.
template <typename T>
__global__ __launch_bounds__(1024) void quantise_long(QuantArgs a) {
  __shared__ float part[16];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint16_t* x = (const uint16_t*)a.X + row * a.ldx;
    float mx = 0.0f;
    for (int64_t j = threadIdx.x * 8; j < a.cols; j += 8192) mx = largest<T>(load8<true>(x, (int)j, a.cols), mx);
    mx = wave::all<MaxBits>(mx);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mx;
    __syncthreads();
    for (int i = 0; i < 16; ++i) mx = MaxBits::op(mx, part[i]);
    const float s = scale_of(mx);
    const float inv = 1.0f / s;
    if (threadIdx.x == 0) a.scale[row] = s;
    for (int64_t j = threadIdx.x * 8; j < a.cols; j += 8192)
      quantise8<T, true>(a.Y + row * a.ldy, (int)j, a.cols, load8<true>(x, (int)j, a.cols), s, inv);
    __syncthreads();  // `part` is free for the next row
  }
}

constexpr int kMaxGrid = 1 << 20;  // a grid's threads fit 32 bits; further rows by the kernels' loops

// What exceeds the L2s' 32 MiB is read past the caches.
bool past_caches(int64_t bytes) { return bytes > (int64_t)32 << 20; }

template <typename T, bool ANY, int VPT, int LPR>
hipError_t launch_quantise(const QuantArgs& a, hipStream_t stream) {
  constexpr int RPB = LPR ? 256 / (LPR + !LPR) : 1;
  const int wgs = (int)(((int64_t)a.rows + RPB - 1) / RPB);
  const int waves = LPR ? 4 : (a.cols + 512 * VPT - 1) / (512 * VPT);
  const dim3 grid(min(wgs, kMaxGrid)), block(64 * waves);
  if (!ANY && past_caches((int64_t)a.rows * a.cols * 2)) hipLaunchKernelGGL((quantise_rows<T, ANY, VPT, LPR, !ANY>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((quantise_rows<T, ANY, VPT, LPR, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}
template <typename T, bool ANY>
hipError_t launch_quantise(const QuantArgs& a, hipStream_t stream) {
  if (a.cols <= 128) return launch_quantise<T, ANY, 1, 16>(a, stream);
  if (a.cols <= 512 || (a.cols <= 8192 && a.rows < 1024)) return launch_quantise<T, ANY, 1, 0>(a, stream);
  if (a.cols <= 16384) return launch_quantise<T, ANY, 2, 0>(a, stream);
  if (a.cols <= 32768) return launch_quantise<T, ANY, 4, 0>(a, stream);
  hipLaunchKernelGGL((quantise_long<T>), dim3(min(a.rows, kMaxGrid)), dim3(1024), 0, stream, a);
  return hipGetLastError();
}
template <typename T>
hipError_t launch_quantise(const QuantArgs& a, hipStream_t stream) {
  const bool aligned = ((a.cols | a.ldx | a.ldy) & 7) == 0 && ((uintptr_t)a.X & 15u) == 0 && ((uintptr_t)a.Y & 7u) == 0;
  return aligned ? launch_quantise<T, false>(a, stream) : launch_quantise<T, true>(a, stream);
}

// ---------------------------------------------------------------------------
// a token's rows brought together
// ---------------------------------------------------------------------------
struct CombineArgs {
  const void *Z, *R;
  void* Y;
  const float* weights;
  const int32_t* ids;
  int64_t ldz, ldr, ldy, tokens;
  int per, experts, cols, chunks;
};

// A workgroup a token and 2048 columns of it, eight a thread, four rows' loads and
// the residual's at a time in flight.
template <typename T, bool ANY, bool PAST>
__global__ __launch_bounds__(256) void combine_rows(CombineArgs a) {
  constexpr int B = 4;
  const int64_t units = a.tokens * a.chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t t = u / a.chunks;
    const int col = (int)(u - t * a.chunks) * 2048 + threadIdx.x * 8;
    float s[8] = {}, f[8];
    u32x4 r = {};
    if (a.R) r = load8<ANY, PAST>((const uint16_t*)a.R + t * a.ldr, col, a.cols);
    for (int j0 = 0; j0 < a.per; j0 += B) {
      u32x4 z[B];
      float w[B];
      bool in[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int64_t q = t * a.per + min(j0 + b, a.per - 1);
        in[b] = j0 + b < a.per && (!a.ids || (uint32_t)a.ids[q] < (uint32_t)a.experts);
        w[b] = a.weights[q];
        if (in[b]) z[b] = load8<ANY, PAST>((const uint16_t*)a.Z + q * a.ldz, col, a.cols);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (!in[b]) continue;
        widen<T>(z[b], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(w[b], f[i], s[i]);
      }
    }
    if (a.R) {
      widen<T>(r, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += f[i];
    }
    store8<T, ANY>((T*)a.Y + t * a.ldy, col, a.cols, s);
  }
}

template <typename T>
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const int64_t lds = a.cols | a.ldz | a.ldy | (a.R ? a.ldr : 0);
  const uintptr_t ptrs = (uintptr_t)a.Z | (uintptr_t)a.R | (uintptr_t)a.Y;
  const dim3 grid((uint32_t)std::min<int64_t>(a.tokens * a.chunks, kMaxGrid));
  if ((lds & 7) != 0 || (ptrs & 15u) != 0) hipLaunchKernelGGL((combine_rows<T, true, false>), grid, dim3(256), 0, stream, a);
  else if (past_caches(a.tokens * a.per * a.cols * 2)) hipLaunchKernelGGL((combine_rows<T, false, true>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((combine_rows<T, false, false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

constexpr int64_t kLim = (int64_t)1 << 31;
constexpr int64_t kMaxCols = (int64_t)1 << 30;  // a thread's column and the eight behind it are 32-bit integers

gemm_epi_status status_of(hipError_t e) {
  if (e == hipSuccess) return GEMM_EPI_OK;
  set_last_hip_error((int)e);
  return GEMM_EPI_ERR_HIP;
}

}  // namespace rows
}  // namespace ge

extern "C" {

gemm_epi_status gemm_epi_quantise_i8(const void* X, int64_t ldx, int8_t* Y, int64_t ldy, float* scale, int64_t rows,
                                     int64_t cols, gemm_epi_dtype dtype, void* stream) {
  using namespace ge::rows;
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_INVALID_ARG;
  if (rows < 0 || cols <= 0 || ldx < cols || ldy < cols || !X || !Y || !scale) return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)X & 1u) || ((uintptr_t)scale & 3u)) return GEMM_EPI_ERR_INVALID_ARG;
  if (rows >= kLim || cols > kMaxCols) return GEMM_EPI_ERR_UNSUPPORTED;
  if (rows == 0) return GEMM_EPI_OK;
  const QuantArgs a{X, Y, scale, ldx, ldy, (int)rows, (int)cols};
  const hipStream_t s = (hipStream_t)stream;
  return status_of(dtype == GEMM_EPI_F16 ? launch_quantise<ge::f16>(a, s) : launch_quantise<ge::bf16>(a, s));
}

gemm_epi_status gemm_epi_combine(const void* Z, int64_t ldz, const float* weights, const int32_t* ids, int64_t experts,
                                 const void* R, int64_t ldr, void* Y, int64_t ldy, int64_t tokens, int64_t per,
                                 int64_t cols, gemm_epi_dtype dtype, void* stream) {
  using namespace ge::rows;
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_INVALID_ARG;
  if (tokens < 0 || per <= 0 || cols <= 0 || experts <= 0 || ldz < cols || ldy < cols || (R && ldr < cols) || !Z ||
      !Y || !weights)
    return GEMM_EPI_ERR_INVALID_ARG;
  if ((((uintptr_t)Z | (uintptr_t)R | (uintptr_t)Y) & 1u) || (((uintptr_t)weights | (uintptr_t)ids) & 3u))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (per > 64 || tokens >= kLim || tokens * per >= kLim || cols > kMaxCols) return GEMM_EPI_ERR_UNSUPPORTED;
  if (tokens == 0) return GEMM_EPI_OK;
  const CombineArgs a{Z,   R,   Y,   weights, ids,      ldz,
                      ldr, ldy, tokens, (int)per, (int)std::min<int64_t>(experts, kLim - 1), (int)cols, (int)((cols + 2047) / 2048)};
  const hipStream_t s = (hipStream_t)stream;
  return status_of(dtype == GEMM_EPI_F16 ? launch_combine<ge::f16>(a, s) : launch_combine<ge::bf16>(a, s));
}

}  // extern "C"
