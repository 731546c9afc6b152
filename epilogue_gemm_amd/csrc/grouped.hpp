// grouped.hpp -- products of rows with the weights of their groups,
//
//     C[.] = act(X[.] W[g]^T + bias[g])   or   act(gate) * up
//
// for 16-bit formats and, with scales, 8-bit integers; one group of all rows
// is the 8-bit product.
#pragma once

#include <algorithm>

#include "gemm_tile16.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_experts.h"

namespace ge {
namespace grouped {

struct Args {
  const int32_t *offsets, *order;  // (no offsets: one group of all rows)
  const void *X, *W, *bias, *R;
  const float *xs, *ws;
  void* C;
  int64_t ldx, ldw, ldr, ldc;  // in elements
  int64_t group_w;             // elements between the groups' weights
  int groups, rows, per, N, K;
  int gather, scatter, epi;
  int tiles_n;
};

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Elem {
  static constexpr bool kInt = __is_same(T, int8_t);
  using acc = std::conditional_t<kInt, i32x4, f32x4>;
};

template <typename T>
__device__ __forceinline__ typename Elem<T>::acc mfma(u32x4 a, u32x4 b, typename Elem<T>::acc c) {
  if constexpr (Elem<T>::kInt)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  else return tile16::mfma16<T>(a, b, c);
}

// ---------------------------------------------------------------------------
// a workgroup's tile
// ---------------------------------------------------------------------------
struct Found {
  int group;       // -1: none
  int begin, end;  // places of the tile's rows
  int tn;
};

// Places of group g, of offsets that may hold anything.
__device__ __forceinline__ int clamped(const Args& a, int g) { return max(0, min(a.offsets[g], a.rows)); }

// Tile `id` of those of all groups, group by group, in each column by column.
// Every wave counts the tiles of the groups for itself, lane l those of groups
// l * per .. + per - 1.
template <int BM>
__device__ __forceinline__ Found find_tile(const Args& a, int id, int lane) {
  if (!a.offsets) {
    const int tiles_m = (a.rows + BM - 1) / BM;
    const int tn = id / tiles_m, m = id - tn * tiles_m;
    return Found{tn < a.tiles_n ? 0 : -1, m * BM, min(a.rows, m * BM + BM), tn};
  }
  const int per = (a.groups + 63) / 64, g0 = min(lane * per, a.groups), g1 = min(g0 + per, a.groups);
  int own = 0;
  for (int g = g0; g < g1; ++g) own += (max(0, clamped(a, g + 1) - clamped(a, g)) + BM - 1) / BM;
  // (offsets that do not ascend may count rows twice: the sum over lanes then
  // wraps, a lane's own does not)
  const uint32_t left = (uint32_t)id - (uint32_t)(wave::scan(own) - own) * (uint32_t)a.tiles_n;
  const uint64_t owner = __builtin_amdgcn_ballot_w64(left < (uint32_t)own * (uint32_t)a.tiles_n);
  if (owner == 0) return Found{-1, 0, 0, 0};
  // its group: the lane that counted it walks there
  int at = (int)left, g = g0, begin = 0, end = 0, tiles = 1;
  for (; g < g1; ++g) {
    begin = clamped(a, g);
    end = clamped(a, g + 1);
    tiles = (max(0, end - begin) + BM - 1) / BM;
    if (at < tiles * a.tiles_n) break;
    at -= tiles * a.tiles_n;
  }
  const int src = __builtin_ctzll(owner);
  g = __builtin_amdgcn_readlane(g, src);
  begin = __builtin_amdgcn_readlane(begin, src);
  end = __builtin_amdgcn_readlane(end, src);
  tiles = __builtin_amdgcn_readlane(tiles, src);
  at = __builtin_amdgcn_readlane(at, src);
  const int tn = at / tiles;
  begin += (at - tn * tiles) * BM;
  return Found{g, begin, min(end, begin + BM), tn};
}

// Entry of place i (-1: none).
__device__ __forceinline__ int entry_of(const Args& a, int i) {
  if (!a.order) return i;
  const int q = a.order[i];
  return (uint32_t)q < (uint32_t)a.rows ? q : -1;
}

// ---------------------------------------------------------------------------
// the outputs
// ---------------------------------------------------------------------------
__device__ __forceinline__ float activated(float z, int epi) {
  switch (epi) {
    case GEMM_EPI_RELU:
    case GEMM_EPI_BIAS_RELU: return fmaxf(z, 0.0f);
    case GEMM_EPI_BIAS_GELU: return gelu_logistic(z);
    case GEMM_EPI_SILU:
    case GEMM_EPI_BIAS_SILU: return silu_logistic(z);
    default: return z;
  }
}
__device__ __forceinline__ bool has_bias(int epi) {
  return epi == GEMM_EPI_BIAS || epi == GEMM_EPI_BIAS_RELU || epi == GEMM_EPI_BIAS_GELU || epi == GEMM_EPI_BIAS_SILU;
}

// Row r of a tile of W: blocks of 16 columns of the output, gated ones of 16
// gates and 16 ups in turn, so that a lane has both of an output.
template <bool GATED>
__device__ __forceinline__ int column_of(int r) {
  return GATED ? (r >> 5) * 16 + (r & 15) : r;
}

// ---------------------------------------------------------------------------
// a simple kernel: tiles of 64 x 64, one stage through registers
// ---------------------------------------------------------------------------
template <typename T, typename TOut, bool GATED>
__global__ __launch_bounds__(256) void simple_kernel(Args a) {
  constexpr int BM = 64, BN = 64, ROW = 128, LD = ROW + 16;
  constexpr int ES = sizeof(T), OUT = GATED ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) char sa[BM * LD], sb[BN * LD];
  __shared__ int xrow[BM], crow[BM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Found f = find_tile<BM>(a, blockIdx.x, lane);
  if (f.group < 0) return;
  if (tid < BM) {
    const int i = f.begin + tid, q = i < f.end ? entry_of(a, i) : -1;
    xrow[tid] = q < 0 ? -1 : a.gather ? q / a.per : i;
    crow[tid] = q < 0 ? -1 : a.scatter ? q : i;
  }
  __syncthreads();
  const int wm = wave >> 1, wn = wave & 1, c = lane & 15, h = lane >> 4;
  typename Elem<T>::acc acc[2][2] = {};
  const char* w = (const char*)a.W + f.group * a.group_w * ES;
  const int64_t row_bytes = (int64_t)a.K * ES;
  for (int64_t k0 = 0; k0 < row_bytes; k0 += ROW) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int piece = tid + 256 * p, r = piece >> 3, at = (piece & 7) * 16;
      u32x4 x = {}, y = {};
      if (k0 + at < row_bytes) {
        if (xrow[r] >= 0) x = *(const u32x4*)((const char*)a.X + xrow[r] * a.ldx * ES + k0 + at);
        const int n = f.tn * OUT + column_of<GATED>(r);
        if (n < a.N) y = *(const u32x4*)(w + (int64_t)(n + (GATED && (r & 16) ? a.N : 0)) * a.ldw * ES + k0 + at);
      }
      *(u32x4*)(sa + r * LD + at) = x;
      *(u32x4*)(sb + r * LD + at) = y;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = mfma<T>(*(const u32x4*)(sb + (wn * 32 + j * 16 + c) * LD + kk * 64 + h * 16),
                              *(const u32x4*)(sa + (wm * 32 + i * 16 + c) * LD + kk * 64 + h * 16), acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wm * 32 + i * 16 + c;
    if (crow[r] < 0) continue;
    const float xs = Elem<T>::kInt ? a.xs[xrow[r]] : 1.0f;
    TOut* out = (TOut*)a.C + crow[r] * a.ldc;
    // the columns of a block of this wave, before the epilogue's end
    auto value = [&](int j, int e, int n) __attribute__((always_inline)) {
      const int64_t at = (int64_t)f.group * a.N * (GATED ? 2 : 1) + (GATED && (j & 1) ? a.N : 0) + n;
      float z = (float)acc[i][j][e];
      if constexpr (Elem<T>::kInt) z = z * xs * a.ws[at];
      return has_bias(a.epi) ? z + to_f32(((const TOut*)a.bias)[at]) : z;
    };
#pragma unroll
    for (int j = 0; j < 2; j += GATED ? 2 : 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = f.tn * OUT + column_of<GATED>(wn * 32 + j * 16) + 4 * h + e;
        if (n >= a.N) continue;
        float v = activated(value(j, e, n), a.epi);
        if constexpr (GATED) v *= value(j + 1, e, n);
        else if (a.R) v += to_f32(((const TOut*)a.R)[crow[r] * a.ldr + n]);
        out[n] = from_f32<TOut>(v);
      }
  }
}

template <typename T, typename TOut>
hipError_t launch(Args a, bool gated, hipStream_t stream) {
  const int cols = gated ? 32 : 64;
  a.tiles_n = (a.N + cols - 1) / cols;
  // tiles of rows of all groups: what their ends can add
  const int64_t tiles_m = a.offsets ? a.rows / 64 + std::min(a.groups, a.rows) : (a.rows + 63) / 64;
  const dim3 grid((uint32_t)(tiles_m * a.tiles_n)), block(256);
  if (gated) hipLaunchKernelGGL((simple_kernel<T, TOut, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((simple_kernel<T, TOut, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// one translation unit per (input, output) format pair
hipError_t launch_f16_f16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_bf16_bf16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_i8_f16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_i8_bf16(const Args& a, bool gated, hipStream_t stream);

}  // namespace grouped
}  // namespace ge
