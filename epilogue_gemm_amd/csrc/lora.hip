// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//     C[m] = R[m] + s[a] (X[m] A[a]^T) B[a]^T        a = ids[m]
//
// Two kernels.  `shrink` forms U = X A^T (rank values a row) as fp32 partial
// sums over ranges of K; `expand` adds the partials in their order, brings
// U to the input format in two parts and multiplies with B.  Rows come in
// any order of adapters: a workgroup takes 16 consecutive rows -- one MFMA
// operand -- and runs once over each adapter that occurs among them, keeping
// of each product the rows that are the adapter's.
#include "gemm_tile16.hpp"

#include "../../include/gemm_epi_decode.h"

namespace ge {
namespace lora {

using tile16::mfma16;

constexpr int kRows = 16;  // rows of a workgroup: one 16x16x32 operand

struct Args {
  const void *X, *A, *B, *R;
  const float* scale;
  const int32_t* ids;
  void* C;
  float* U;  // [ksplit][M][rank rounded up to 16]
  int64_t ldx, ldr, ldc;
  int M, N, K, rank, adapters;
  int ksplit, kper;  // ranges of K, and their length (a multiple of 128)
  bool vec;          // C and R by 16-byte accesses
};

// The adapter of this lane's row (row = lane % 16), -1 for none.
__device__ __forceinline__ int row_adapter(const Args& a, int row) {
  const int id = row < a.M ? a.ids[row] : -1;
  return id >= 0 && id < a.adapters ? id : -1;
}

// f(adapter, lanes) for each adapter among the 16 rows, in the order of
// their first rows; uniform over the wave.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F&& f) {
  uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(id >= 0) & 0xffffu;
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t same = (uint32_t)__builtin_amdgcn_ballot_w64(id == a) & 0xffffu;
    todo &= ~same;
    f(a, same);
  }
}

// U^T = A X^T: first operand 16 of the adapter's rows, second the 16 rows of
// X, so that lane (m = l % 16, h = l / 16) receives U[m][16 t + 4 h + e].
// Workgroup (tile, range, z) takes the adapters number z, z + Z, ... of its
// rows; its four waves take every fourth 32-deep step and add up in LDS.
template <typename T, int RT>
__global__ __launch_bounds__(256) void shrink(Args a) {
  constexpr int RP = 16 * RT;
  __shared__ float red[4][kRows][RP + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * kRows;
  const int id = row_adapter(a, row0 + c);
  const T* x = (const T*)a.X + (int64_t)min(row0 + c, a.M - 1) * a.ldx;
  const int kbeg = blockIdx.y * a.kper, kend = min(a.K, kbeg + a.kper);
  int u = 0;
  each_adapter(id, [&](int ad, uint32_t same) {
    if (u++ % gridDim.z != blockIdx.z) return;
    const T* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
      ar[t] = (const T*)a.A + ((int64_t)ad * a.rank + min(16 * t + c, a.rank - 1)) * a.K;
    f32x4 acc[RT] = {};
    for (int k0 = kbeg + 32 * wave; k0 < kend; k0 += 128) {
      const int k = k0 + 8 * h;
      const bool in = k < kend;
      const u32x4 xf = in ? *(const u32x4*)(x + k) : u32x4{};
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const u32x4 af = in ? *(const u32x4*)(ar[t] + k) : u32x4{};
        acc[t] = mfma16<T>(af, xf, acc[t]);
      }
    }
    __syncthreads();  // the last adapter's sums have been read
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][c][16 * t + 4 * h + e] = acc[t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * RP; i += 256) {
      const int m = i / RP, r = i % RP;
      if (same >> m & 1)
        a.U[((int64_t)blockIdx.y * a.M + row0 + m) * RP + r] =
            (red[0][m][r] + red[1][m][r]) + (red[2][m][r] + red[3][m][r]);
    }
  });
}

// C^T = B U^T: first operand 16 rows of B (columns of C), second the 16 rows
// of U, so that lane (m, h) receives four columns of row m per product.  The
// rows of B are fed to the four products of 64 columns so that a lane's are
// 16 consecutive columns.  U, which bounds the result's error, is scaled by a
// power of two so that its row's largest value lies in [1/2, 1) and enters
// as two 16-bit parts, the rounded value and its rounded remainder.
template <typename T, int RT>
__global__ __launch_bounds__(256) void expand(Args a) {
  constexpr int RP = 16 * RT, ST = (RP + 31) / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int row = blockIdx.x * kRows + c;
  const int n0 = (blockIdx.y * 4 + wave) * 64;
  if (n0 >= a.N) return;
  const int id = row_adapter(a, row);
  float u[ST][8];
  float mx = 0.0f;
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const int r = 32 * s + 8 * h;
#pragma unroll
    for (int i = 0; i < 8; ++i) u[s][i] = 0.0f;
    if (id >= 0 && r < a.rank)
      for (int p = 0; p < a.ksplit; ++p) {
        const float* up = a.U + ((int64_t)p * a.M + row) * RP + r;
        const f32x4 lo = *(const f32x4*)up, hi = *(const f32x4*)(up + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[s][i] += lo[i];
          u[s][4 + i] += hi[i];
        }
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(u[s][i]));
  }
  mx = fmaxf(mx, __shfl_xor(mx, 16));
  mx = fmaxf(mx, __shfl_xor(mx, 32));
  // 2^-ex brings mx into [1/2, 1); an infinite or zero row is left as it is
  int ex = mx > 0.0f && mx < __builtin_inff() ? __builtin_amdgcn_frexp_expf(mx) : 0;
  ex = max(ex, -120);
  u32x4 uh[ST], ul[ST];
#pragma unroll
  for (int s = 0; s < ST; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = __builtin_amdgcn_ldexpf(u[s][2 * i], -ex), v1 = __builtin_amdgcn_ldexpf(u[s][2 * i + 1], -ex);
      const T t0 = from_f32<T>(v0), t1 = from_f32<T>(v1);
      const float d0 = v0 - to_f32(t0), d1 = v1 - to_f32(t1);
      uh[s][i] = (uint32_t)bits16(t0) | (uint32_t)bits16(t1) << 16;
      // (the remainder of an infinity is no number: it has none)
      ul[s][i] = pack2_out<T>(fabsf(v0) < __builtin_inff() ? d0 : 0.0f, fabsf(v1) < __builtin_inff() ? d1 : 0.0f);
    }
  f32x4 out[4] = {};
  each_adapter(id, [&](int ad, uint32_t) {
    const T* b = (const T*)a.B + (int64_t)ad * a.N * a.rank;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), a.N - 1);
      f32x4 acc = {};
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const int r = 32 * s + 8 * h;
        const u32x4 bf = r < a.rank ? *(const u32x4*)(b + (int64_t)n * a.rank + r) : u32x4{};
        acc = mfma16<T>(bf, uh[s], acc);
        acc = mfma16<T>(bf, ul[s], acc);
      }
      if (id == ad) out[j] = acc;
    }
  });
  if (row >= a.M) return;
  const float back = id < 0 ? 0.0f : (a.scale ? a.scale[id] : 1.0f);
  const int n = n0 + 16 * h;
  T* cp = (T*)a.C + (int64_t)row * a.ldc;
  const T* rp = a.R ? (const T*)a.R + (int64_t)row * a.ldr : nullptr;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = id < 0 ? 0.0f : __builtin_amdgcn_ldexpf(out[2 * p + (i >> 2)][i & 3], ex) * back;
    const int np = n + 8 * p;
    if (a.vec && np + 8 <= a.N) {
      if (rp) {
        const f32x4 r0 = load4(rp + np), r1 = load4(rp + np + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] += r0[i];
          v[4 + i] += r1[i];
        }
      }
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack2_out<T>(v[2 * i], v[2 * i + 1]);
      *(u32x4*)(cp + np) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (np + i < a.N) cp[np + i] = from_f32<T>(v[i] + (rp ? to_f32(rp[np + i]) : 0.0f));
    }
  }
}

// Ranges of K: enough workgroups for the chip (512), each range at least two
// steps of its four waves.  Depends on the sizes alone.
struct Split {
  int ksplit, kper;
};
inline Split split_k(int64_t M, int64_t K) {
  const int64_t tiles = (M + kRows - 1) / kRows;
  int64_t ks = tiles >= 512 ? 1 : 512 / tiles;
  const int64_t most = (K + 255) / 256;
  if (ks > most) ks = most;
  if (ks > 64) ks = 64;
  const int64_t kper = ((K + ks - 1) / ks + 127) / 128 * 128;
  return Split{(int)((K + kper - 1) / kper), (int)kper};
}

inline int64_t rank_pad(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

template <typename T, int RT>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int tiles = (a.M + kRows - 1) / kRows;
  const int z = min(min(a.adapters, kRows), a.M);
  hipLaunchKernelGGL((shrink<T, RT>), dim3(tiles, a.ksplit, z), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((expand<T, RT>), dim3(tiles, (a.N + 255) / 256), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_rank(const Args& a, hipStream_t stream) {
  switch (rank_pad(a.rank)) {
    case 16: return launch<T, 1>(a, stream);
    case 32: return launch<T, 2>(a, stream);
    case 64: return launch<T, 4>(a, stream);
    default: return launch<T, 8>(a, stream);
  }
}

constexpr int64_t kLim = (int64_t)1 << 31;

// The sizes a call would run (M = 0 included).
gemm_epi_status check_sizes(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters) {
  if (M < 0 || N <= 0 || K <= 0 || rank <= 0 || adapters <= 0) return GEMM_EPI_ERR_INVALID_ARG;
  if (rank > 128 || rank % 8 != 0 || K % 8 != 0 || M >= kLim / 8 || K > kLim - 256 || adapters > 65535 ||
      N > (int64_t)65535 * 256)
    return GEMM_EPI_ERR_UNSUPPORTED;
  return GEMM_EPI_OK;
}

size_t workspace_bytes(int64_t M, int64_t K, int64_t rank) {
  return (size_t)split_k(M, K).ksplit * (size_t)M * (size_t)rank_pad(rank) * 4;
}

}  // namespace lora
}  // namespace ge

extern "C" {

size_t gemm_epi_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t rank, int64_t adapters) {
  if (ge::lora::check_sizes(M, N, K, rank, adapters) != GEMM_EPI_OK || M == 0) return 0;
  return ge::lora::workspace_bytes(M, K, rank);
}

gemm_epi_status gemm_epi_lora(const void* X, int64_t ldx, const void* A, const void* B, const float* scale,
                              const int32_t* ids, const void* R, int64_t ldr, void* C, int64_t ldc, int64_t M,
                              int64_t N, int64_t K, int64_t rank, int64_t adapters, gemm_epi_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || K <= 0 || rank <= 0 || adapters <= 0) return GEMM_EPI_ERR_INVALID_ARG;
  if (ldx < K || ldc < N || (R && ldr < N)) return GEMM_EPI_ERR_INVALID_ARG;
  const gemm_epi_status chk = ge::lora::check_sizes(M, N, K, rank, adapters);
  if (chk != GEMM_EPI_OK) return chk;
  if (M == 0) return GEMM_EPI_OK;
  if (!X || !A || !B || !ids || !C || !workspace) return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)C | (uintptr_t)R) & 1u || ((uintptr_t)ids | (uintptr_t)scale) & 3u) return GEMM_EPI_ERR_INVALID_ARG;
  if (ldx % 8 != 0 || (((uintptr_t)X | (uintptr_t)A | (uintptr_t)B | (uintptr_t)workspace) & 15u))
    return GEMM_EPI_ERR_UNSUPPORTED;
  if (workspace_bytes < ge::lora::workspace_bytes(M, K, rank)) return GEMM_EPI_ERR_INVALID_ARG;
  const ge::lora::Split sp = ge::lora::split_k(M, K);
  const bool vec = (((uintptr_t)C | (uintptr_t)R) & 15u) == 0 && ldc % 8 == 0 && (!R || ldr % 8 == 0);
  const ge::lora::Args a{X,   A,   B,   R,      scale,  ids,       C,           (float*)workspace,
                         ldx, ldr, ldc, (int)M, (int)N, (int)K,    (int)rank,   (int)adapters,
                         sp.ksplit, sp.kper, vec};
  const hipError_t e = dtype == GEMM_EPI_F16 ? ge::lora::launch_rank<ge::f16>(a, (hipStream_t)stream)
                                             : ge::lora::launch_rank<ge::bf16>(a, (hipStream_t)stream);
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}

}  // extern "C"
