// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//     C[m] = R[m] + s[a] (X[m] A[a]^T) B[a]^T        a = ids[m]
//
// Two kernels.  `shrink` forms U = X A^T (rank values a row) as fp32 partial
// sums over ranges of K; `expand` adds the partials in their order, brings
// U to the input format in two parts and multiplies with B.  Rows come in
// any order of adapters: a workgroup takes 16 or 32 consecutive rows -- MFMA
// operands -- and runs once over each adapter that occurs among them, keeping
// of each product the rows that are the adapter's.  Few rows: the adapters
// of a tile are spread over workgroups (grid z), K over more ranges.
#include "gemm_tile16.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_decode.h"

namespace ge {
namespace lora {

using tile16::mfma16;

struct Args {
  const void *X, *A, *B, *R;
  const float* scale;
  const int32_t* ids;
  void* C;
  float* U;  // [ksplit][M][rank rounded up to 16 RT]
  int64_t ldx, ldr, ldc;
  int M, N, K, rank, adapters;
  int ksplit, kper;  // ranges of K, and their length
  bool vec;          // C and R by 16-byte accesses
};

// The adapter of a row, -1 for none.
__device__ __forceinline__ int row_adapter(const Args& a, int row) {
  const int id = row < a.M ? a.ids[row] : -1;
  return id >= 0 && id < a.adapters ? id : -1;
}

// f(adapter, rows) for each adapter among the 16 MT rows from row0 on, in the
// order of their first rows, rows a bit mask; uniform over the wave.
template <int MT, typename F>
__device__ __forceinline__ void each_adapter(const Args& a, int row0, int lane, F&& f) {
  const int id = row_adapter(a, row0 + (lane & (16 * MT - 1)));
  constexpr uint32_t all = MT == 1 ? 0xffffu : 0xffffffffu;
  uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(id >= 0) & all;
  while (todo) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t rows = (uint32_t)__builtin_amdgcn_ballot_w64(id == ad) & all;
    todo &= ~rows;
    f(ad, rows);
  }
}

// U^T = A X^T: first operand 16 of the adapter's rows, second 16 rows of X,
// so that lane (m = l % 16, h = l / 16) receives U[m][16 t + 4 h + e].
// Workgroup (tile, range, z) takes the adapters number z, z + Z, ... of its
// rows; its NW waves take every NW-th 32-deep step and add up in LDS.
// Bound by X (and, for few rows, the adapters) from memory: UNR steps' loads
// are in flight together.
template <typename T, int RT, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void shrink(Args a) {
  constexpr int RP = 16 * RT, ROWS = 16 * MT, UNR = RT + MT > 8 ? 1 : RT + MT > 3 ? 2 : 4;
  __shared__ float red[NW][ROWS][RP + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * ROWS;
  const T* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = (const T*)a.X + (int64_t)min(row0 + 16 * i + c, a.M - 1) * a.ldx + 8 * h;
  const int kbeg = blockIdx.y * a.kper, kend = min(a.K, kbeg + a.kper);
  uint32_t number = 0;
  each_adapter<MT>(a, row0, lane, [&](int ad, uint32_t rows) {
    if (number++ % gridDim.z != blockIdx.z) return;
    const T* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
      ar[t] = (const T*)a.A + ((int64_t)ad * a.rank + min(16 * t + c, a.rank - 1)) * a.K + 8 * h;
    f32x4 acc[MT][RT] = {};
    int k0 = kbeg + 32 * wave;
    for (; k0 + 32 * NW * (UNR - 1) + 32 <= kend; k0 += 32 * NW * UNR) {
      u32x4 xf[UNR][MT], af[UNR][RT];
#pragma unroll
      for (int n = 0; n < UNR; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i) xf[n][i] = *(const u32x4*)(x[i] + k0 + 32 * NW * n);
#pragma unroll
        for (int t = 0; t < RT; ++t) af[n][t] = *(const u32x4*)(ar[t] + k0 + 32 * NW * n);
      }
#pragma unroll
      for (int n = 0; n < UNR; ++n)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[i][t] = mfma16<T>(af[n][t], xf[n][i], acc[i][t]);
    }
    for (; k0 < kend; k0 += 32 * NW) {
      const bool in = k0 + 8 * h < kend;
      u32x4 xf[MT], af[RT];
#pragma unroll
      for (int i = 0; i < MT; ++i) xf[i] = in ? *(const u32x4*)(x[i] + k0) : u32x4{};
#pragma unroll
      for (int t = 0; t < RT; ++t) af[t] = in ? *(const u32x4*)(ar[t] + k0) : u32x4{};
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[i][t] = mfma16<T>(af[t], xf[i], acc[i][t]);
    }
    __syncthreads();  // the last adapter's sums have been read
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[wave][16 * i + c][16 * t + 4 * h + e] = acc[i][t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * RP; i += 64 * NW) {
      const int m = i / RP, r = i % RP;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += red[w][m][r];
      if (rows >> m & 1) a.U[((int64_t)blockIdx.y * a.M + row0 + m) * RP + r] = sum;
    }
  });
}

// C^T = B U^T: first operand 16 rows of B (columns of C), second 16 rows of
// U, so that lane (m, h) receives four columns of row m per product.  The
// rows of B are fed to the four products of a wave's 64 columns so that a
// lane has columns 32 p + 8 h .. + 7 (p = 0, 1): 16-byte pieces of R and C.
// The workgroup first adds up its rows' partials, eight values a thread, and
// leaves U in LDS in two 16-bit parts: scaled by a power of two that brings
// its row's largest value into [1/2, 1), the rounded value and its rounded
// remainder (U's error is the result's).  Then each wave takes every fourth
// 64 columns of the workgroup's.  Bound by R and C (for few rows: by B), U
// and B being small or in the caches.
template <typename T, int RT, int MT>
__global__ __launch_bounds__(256) void expand(Args a) {
  constexpr int RP = 16 * RT, ST = (RP + 31) / 32, ROWS = 16 * MT;
  constexpr int PIECES = RP / 8, LD = RP + 8;  // of a row; a row in LDS
  __shared__ __attribute__((aligned(16))) uint16_t su[2][ROWS][LD];
  __shared__ int sex[ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * ROWS;
  // the rows of the adapters that are this workgroup's; those without one are
  // the first workgroup's
  uint32_t mine = 0;
  {
    uint32_t number = 0, some = 0;
    each_adapter<MT>(a, row0, lane, [&](int, uint32_t rows) {
      some |= rows;
      if (number++ % gridDim.z == blockIdx.z) mine |= rows;
    });
    if (mine == 0 && blockIdx.z != 0) return;
    if (blockIdx.z == 0) mine |= ~some;
  }
#pragma unroll
  for (int i0 = 0; i0 < ROWS * PIECES; i0 += 256) {
    const int i = i0 + threadIdx.x, m = i / PIECES, r = i % PIECES * 8;
    if (ROWS * PIECES % 256 != 0 && i >= ROWS * PIECES) break;
    const int row = row0 + m;
    float u[8] = {};
    if (r < a.rank && row < a.M && (mine >> m & 1)) {
      const float* up = a.U + (int64_t)row * RP + r;
#pragma unroll 8
      for (int p = 0; p < a.ksplit; ++p) {
        const f32x4 lo = *(const f32x4*)(up + (int64_t)p * a.M * RP), hi = *(const f32x4*)(up + (int64_t)p * a.M * RP + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] += lo[e];
          u[4 + e] += hi[e];
        }
      }
    }
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(u[e]));
#pragma unroll
    for (int d = 1; d < PIECES; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    // (an infinite or zero row is left as it is)
    const int ex = mx > 0.0f && mx < __builtin_inff() ? max(__builtin_amdgcn_frexp_expf(mx), -120) : 0;
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v0 = __builtin_amdgcn_ldexpf(u[2 * e], -ex), v1 = __builtin_amdgcn_ldexpf(u[2 * e + 1], -ex);
      const T t0 = from_f32<T>(v0), t1 = from_f32<T>(v1);
      hi[e] = (uint32_t)bits16(t0) | (uint32_t)bits16(t1) << 16;
      // (the remainder of an infinity is no number: it has none)
      lo[e] = pack2_out<T>(fabsf(v0) < __builtin_inff() ? v0 - to_f32(t0) : 0.0f,
                           fabsf(v1) < __builtin_inff() ? v1 - to_f32(t1) : 0.0f);
    }
    *(u32x4*)&su[0][m][r] = hi;
    *(u32x4*)&su[1][m][r] = lo;
    if (r == 0) sex[m] = ex;
  }
  __syncthreads();
  int id[MT], ex[MT];
  u32x4 uh[MT][ST], ul[MT][ST];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    id[i] = row_adapter(a, row0 + 16 * i + c);
    ex[i] = sex[16 * i + c];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      const int r = 32 * s + 8 * h;
      uh[i][s] = r < RP ? *(const u32x4*)&su[0][16 * i + c][r] : u32x4{};
      ul[i][s] = r < RP ? *(const u32x4*)&su[1][16 * i + c][r] : u32x4{};
    }
  }
  for (int n0 = (blockIdx.y * 4 + wave) * 64; n0 < a.N; n0 += gridDim.y * 256) {
    // R's pieces first: nothing depends on them until the end
    u32x4 rr[MT][2];
    const bool vec = a.vec && n0 + 64 <= a.N;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        rr[i][p] = vec && a.R && row0 + 16 * i + c < a.M
                       ? *(const u32x4*)((const T*)a.R + (int64_t)(row0 + 16 * i + c) * a.ldr + n0 + 32 * p + 8 * h)
                       : u32x4{};
    f32x4 out[MT][4] = {};
    each_adapter<MT>(a, row0, lane, [&](int ad, uint32_t rows) {
      if ((rows & mine) == 0) return;
      const T* b = (const T*)a.B + (int64_t)ad * a.N * a.rank;
      u32x4 bf[4][ST];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = min(n0 + 32 * (j >> 1) + 8 * (c >> 2) + 4 * (j & 1) + (c & 3), a.N - 1);
#pragma unroll
        for (int s = 0; s < ST; ++s) {
          const int r = 32 * s + 8 * h;
          bf[j][s] = r < a.rank ? *(const u32x4*)(b + (int64_t)n * a.rank + r) : u32x4{};
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 acc = {};
#pragma unroll
          for (int s = 0; s < ST; ++s) {
            acc = mfma16<T>(bf[j][s], uh[i][s], acc);
            acc = mfma16<T>(bf[j][s], ul[i][s], acc);
          }
          if (id[i] == ad) out[i][j] = acc;
        }
    });
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = row0 + 16 * i + c;
      if (row >= a.M || !(mine >> (16 * i + c) & 1)) continue;
      const float back = id[i] >= 0 && a.scale ? a.scale[id[i]] : 1.0f;
      T* cp = (T*)a.C + (int64_t)row * a.ldc;
      const T* rp = a.R ? (const T*)a.R + (int64_t)row * a.ldr : nullptr;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int n = n0 + 32 * p + 8 * h;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = id[i] < 0 ? 0.0f : __builtin_amdgcn_ldexpf(out[i][2 * p + (e >> 2)][e & 3], ex[i]) * back;
        if (vec) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float r0 = to_f32(__builtin_bit_cast(T, (uint16_t)(rr[i][p][e] & 0xffffu)));
            const float r1 = to_f32(__builtin_bit_cast(T, (uint16_t)(rr[i][p][e] >> 16)));
            w[e] = pack2_out<T>(v[2 * e] + r0, v[2 * e + 1] + r1);
          }
          *(u32x4*)(cp + n) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) cp[n + e] = from_f32<T>(v[e] + (rp ? to_f32(rp[n + e]) : 0.0f));
        }
      }
    }
  }
}

// How a problem is cut, by its sizes alone.  Many rows (from 1024): 32 of
// them share an adapter's values (MT = 2), eight waves add up a range.
struct Cut {
  int mt, nw, tiles, ksplit, kper;
};
inline Cut cut(int64_t M, int64_t K) {
  Cut s;
  s.mt = M >= 1024 ? 2 : 1;
  s.nw = 4 * s.mt;
  s.tiles = (int)((M + 16 * s.mt - 1) / (16 * s.mt));
  // ranges of K: some 256 workgroups, two steps of its waves or more each
  const int step = 32 * s.nw;
  int64_t ks = s.tiles >= 256 ? 1 : 256 / s.tiles;
  const int64_t most = (K + 2 * step - 1) / (2 * step);
  if (ks > most) ks = most;
  s.kper = (int)(((K + ks - 1) / ks + step - 1) / step * step);
  s.ksplit = (int)((K + s.kper - 1) / s.kper);
  return s;
}

inline int64_t rank_pad(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

template <typename T, int RT, int MT>
hipError_t launch(const Args& a, const Cut& s, hipStream_t stream) {
  // workgroups among which a tile's adapters are spread: as many as it can
  // hold where tiles are few
  const int z = min(min(a.adapters, a.M), s.tiles <= 4 ? 16 : s.tiles <= 256 ? 4 : 1);
  // columns of a workgroup: 256 each, or more where that still leaves 512
  // workgroups, so that U is read and split less often
  const int chunks = (a.N + 255) / 256, y = min(chunks, max(1, 512 / s.tiles));
  hipLaunchKernelGGL((shrink<T, RT, MT, 4 * MT>), dim3(s.tiles, s.ksplit, z), dim3(256 * MT), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((expand<T, RT, MT>), dim3(s.tiles, y, z), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T, int RT>
hipError_t launch(const Args& a, const Cut& s, hipStream_t stream) {
  return s.mt == 2 ? launch<T, RT, 2>(a, s, stream) : launch<T, RT, 1>(a, s, stream);
}

template <typename T>
hipError_t launch_rank(const Args& a, const Cut& s, hipStream_t stream) {
  switch (rank_pad(a.rank)) {
    case 16: return launch<T, 1>(a, s, stream);
    case 32: return launch<T, 2>(a, s, stream);
    case 64: return launch<T, 4>(a, s, stream);
    default: return launch<T, 8>(a, s, stream);
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
  return (size_t)cut(M, K).ksplit * (size_t)M * (size_t)rank_pad(rank) * 4;
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
  const ge::lora::Cut cut = ge::lora::cut(M, K);
  const bool vec = (((uintptr_t)C | (uintptr_t)R) & 15u) == 0 && ldc % 8 == 0 && (!R || ldr % 8 == 0);
  const ge::lora::Args a{X,   A,   B,   R,      scale,  ids,       C,           (float*)workspace,
                         ldx, ldr, ldc, (int)M, (int)N, (int)K,    (int)rank,   (int)adapters,
                         cut.ksplit, cut.kper, vec};
  const hipError_t e = dtype == GEMM_EPI_F16 ? ge::lora::launch_rank<ge::f16>(a, cut, (hipStream_t)stream)
                                             : ge::lora::launch_rank<ge::bf16>(a, cut, (hipStream_t)stream);
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}

}  // extern "C"
