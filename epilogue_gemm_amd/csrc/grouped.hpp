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

// A tile of those of all groups, from the workgroup's number.  Workgroups go to
// the 8 XCDs in turn: consecutive tiles go to one XCD, group by group, in each
// in panels of PANEL tiles of rows, column by column, so that the tiles which
// one XCD works on together share rows of X and of W in its L2.  Every wave
// counts the tiles of the groups for itself, lane l those of groups l * per ..
// + per - 1.
template <int BM, int PANEL>
__device__ __forceinline__ Found find_tile(const Args& a, int id, int lane) {
  int own = 0, g0 = 0, g1 = 0, incl = 0, total;
  if (a.offsets) {
    const int per = (a.groups + 63) / 64;
    g0 = min(lane * per, a.groups);
    g1 = min(g0 + per, a.groups);
    for (int g = g0; g < g1; ++g) own += (max(0, clamped(a, g + 1) - clamped(a, g)) + BM - 1) / BM;
    // (offsets that do not ascend may count rows twice: the sum over lanes then
    // wraps, a lane's own does not)
    incl = wave::scan(own);
    total = __builtin_amdgcn_readlane(incl, 63);
  } else {
    total = (a.rows + BM - 1) / BM;
  }
  const uint32_t all = (uint32_t)total * (uint32_t)a.tiles_n;
  if ((uint32_t)id >= all) return Found{-1, 0, 0, 0};
  const uint32_t x = id & 7, f = x * (all >> 3) + min(x, all & 7) + ((uint32_t)id >> 3);
  int g = 0, begin = 0, end = a.rows, tiles = total, at = (int)f;
  if (a.offsets) {
    const uint32_t left = f - (uint32_t)(incl - own) * (uint32_t)a.tiles_n;
    const uint64_t owner = __builtin_amdgcn_ballot_w64(left < (uint32_t)own * (uint32_t)a.tiles_n);
    if (owner == 0) return Found{-1, 0, 0, 0};
    // its group: the lane that counted it walks there
    at = (int)left;
    tiles = 1;
    for (g = g0; g < g1; ++g) {
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
  }
  const int p = at / (PANEL * a.tiles_n), r = at - p * (PANEL * a.tiles_n), high = min(PANEL, tiles - p * PANEL);
  const int tn = r / high;
  begin += (p * PANEL + r - tn * high) * BM;
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
// f(an epilogue without a bias, as a constant) of the activation of `epi`.
template <typename F>
__device__ __forceinline__ void with_activation(int epi, F&& f) {
  if (epi == GEMM_EPI_NONE || epi == GEMM_EPI_BIAS) f(std::integral_constant<int, GEMM_EPI_NONE>{});
  else if (epi == GEMM_EPI_RELU || epi == GEMM_EPI_BIAS_RELU) f(std::integral_constant<int, GEMM_EPI_RELU>{});
  else if (epi == GEMM_EPI_BIAS_GELU) f(std::integral_constant<int, GEMM_EPI_BIAS_GELU>{});
  else f(std::integral_constant<int, GEMM_EPI_SILU>{});
}
// of z, which has its bias
template <int ACT>
__device__ __forceinline__ float activated(float z) {
  return epilogue<ACT>(z, 0.0f);
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
  const Found f = find_tile<BM, 4>(a, blockIdx.x, lane);
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
  with_activation(a.epi, [&](auto act) __attribute__((always_inline)) {
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
        float v = activated<decltype(act)::value>(value(j, e, n));
        if constexpr (GATED) v *= value(j + 1, e, n);
        else if (a.R) v += to_f32(((const TOut*)a.R)[crow[r] * a.ldr + n]);
        out[n] = from_f32<TOut>(v);
      }
  }  });
}

// ---------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------
using tile::kRowBytes;
using tile::lds_ptr;

// Direct copies of a tile's rows into LDS, 128 bytes of K a k-step, in the
// layout of gemm_tile16.hpp: instruction i of wave w (of NW) fills rows (NW i +
// w) * 8 .. + 7, 16-byte chunk c of row r at position c ^ (r & 7).  The rows
// may lie anywhere in the buffer: a lane keeps the offset of its row for each
// instruction, past the buffer's end (zeros, no access) for a row that is none.
// The k axis is shifted by `pad` bytes, so that the last k-steps are whole and
// the chunks of the first before K's beginning load as zeros.
template <int R, int NW>
struct RowLoader {
  static constexpr int NI = R / (8 * NW);
  static_assert(NI >= 1 && NI <= 8 && R % (8 * NW) == 0, "whole instructions");
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t voff[8];  // fixed extent: one by NI left host kernel stubs undefined
  int wave, chunk;

  // row(r): the bytes from `base` to tile row r, or a negative number
  template <typename F>
  __device__ __forceinline__ RowLoader(const char* base, int64_t bytes, int pad, int tid, F&& row) {
    rsrc = tile::make_rsrc(base - pad, (uint32_t)min(bytes + pad, (int64_t)0xfffff000));
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t at = row((NW * i + wave) * 8 + (lane >> 3));
      voff[i] = at < 0 ? 0xFFFFFFF0u : (uint32_t)at + 16 * chunk;
    }
  }
  __device__ __forceinline__ void issue(char* dst, int kt, int i) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(dst + (NW * i + wave) * 1024), 16, voff[i],
                                             kt * kRowBytes, 0, 0);
  }
  __device__ __forceinline__ void issue_first(char* dst, int kt, int i, int pad) const {
    const uint32_t v = 16 * chunk + kt * kRowBytes < pad ? 0xFFFFFFF0u : voff[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(dst + (NW * i + wave) * 1024), 16, v, kt * kRowBytes, 0, 0);
  }
};

// What the epilogue needs of a tile's rows and columns, in LDS.
template <int BM, int BN>
struct Edges {
  int c[BM];      // row of C, -1: none
  float xs[BM];   // a row's scale (8-bit rows)
  f32x4 ws[BN / 4], bias[BN / 4];  // of each row of the tile of W
};

// The tile's rows of X, -1 for none, are left in xrow.
template <typename T, typename TOut, bool GATED, int BM, int BN>
__device__ __forceinline__ void fill_edges(const Args& a, const Found& f, Edges<BM, BN>& edges, int* xrow, int tid, int threads) {
  for (int r = tid; r < BM; r += threads) {
    const int i = f.begin + r, q = i < f.end ? entry_of(a, i) : -1, x = q < 0 ? -1 : a.gather ? q / a.per : i;
    xrow[r] = x;
    edges.c[r] = q < 0 ? -1 : a.scatter ? q : i;
    if constexpr (Elem<T>::kInt) edges.xs[r] = q < 0 ? 0.0f : a.xs[x];
  }
  const bool biased = has_bias(a.epi);
  for (int r = tid; r < BN; r += threads) {
    const int n = f.tn * (GATED ? BN / 2 : BN) + column_of<GATED>(r);
    const int64_t at = (int64_t)f.group * a.N * (GATED ? 2 : 1) + (GATED && (r & 16) ? a.N : 0) + n;
    if constexpr (Elem<T>::kInt) ((float*)edges.ws)[r] = n < a.N ? a.ws[at] : 0.0f;
    ((float*)edges.bias)[r] = biased && n < a.N ? to_f32(((const TOut*)a.bias)[at]) : 0.0f;
  }
}

// Epilogue of a wave's TM x TN blocks of 16 x 16 (lane (c, h) has columns 4 h
// .. + 3 of row c of each), rows r0 .. and W's rows w0 .. of the tile, output
// columns n0 ..: the scales, bias, activation, gate's product or residual in
// fp32, one rounding, then each band of 16 rows through the wave's own LDS
// (16-byte chunks swizzled by row) and out in 16-byte pieces along rows.
template <typename T, typename TOut, bool GATED, int ACT, int TM, int TN, int BM, int BN>
__device__ __forceinline__ void write_rows(const Args& a, const typename Elem<T>::acc (&acc)[TM][TN],
                                           const Edges<BM, BN>& edges, int r0, int w0, int n0, int lane, char* stage) {
  constexpr int W = (GATED ? TN / 2 : TN) * 16;   // output columns
  constexpr int CPR = W * 2 / 16, SWM = (CPR < 16 ? CPR : 16) - 1, RPI = 64 / CPR < 16 ? 64 / CPR : 16;
  constexpr int S = GATED ? 2 : 1;
  const int c = lane & 15, h = lane >> 4;
  static_for<TM>([&](auto i_c) __attribute__((always_inline)) {
    constexpr int i = decltype(i_c)::value;
    const int row = r0 + 16 * i;
    const float xs = Elem<T>::kInt ? edges.xs[row + c] : 1.0f;
    const int to = edges.c[row + c];
    static_for<TN / S>([&](auto j_c) __attribute__((always_inline)) {
      constexpr int j = decltype(j_c)::value;
      auto z = [&](auto jj_c) __attribute__((always_inline)) {
        constexpr int jj = decltype(jj_c)::value;
        const int at = w0 / 4 + 4 * jj + h;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][jj][e];
        if constexpr (Elem<T>::kInt) v = v * xs * edges.ws[at];
        return v + edges.bias[at];
      };
      const int n = n0 + j * 16 + 4 * h;
      f32x4 v = z(std::integral_constant<int, S * j>{});
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = activated<ACT>(v[e]);
      if constexpr (GATED) {
        v *= z(std::integral_constant<int, 2 * j + 1>{});
      } else if (a.R && to >= 0) {
        const TOut* r = (const TOut*)a.R + to * a.ldr + n;
        if (n + 4 <= a.N && ((uintptr_t)r & 7u) == 0) {
          v += load4<TOut>(r);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) v[e] += to_f32(r[e]);
        }
      }
      const int chunk = 2 * j + (h >> 1);
      *(u32x2*)(stage + c * (W * 2) + ((chunk ^ (c & SWM)) << 4) + 8 * (h & 1)) =
          u32x2{pack2_out<TOut>(v[0], v[1]), pack2_out<TOut>(v[2], v[3])};
    });
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS accesses are done in order)
#pragma unroll
    for (int t = 0; t < 16 / RPI; ++t) {
      const int r = t * RPI + lane / CPR, ch = lane % CPR;
      if (RPI * CPR < 64 && lane >= RPI * CPR) continue;
      const u32x4 d = *(const u32x4*)(stage + r * (W * 2) + ((ch ^ (r & SWM)) << 4));
      const int cr = edges.c[row + r], n = n0 + 8 * ch;
      if (cr < 0 || n >= a.N) continue;
      uint16_t* dst = (uint16_t*)a.C + cr * a.ldc + n;
      if (n + 8 <= a.N && ((uintptr_t)dst & 15u) == 0) {
        *(u32x4*)dst = d;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.N) dst[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  });
}

// BM x BN products (BN / 2 gated outputs) by 2 x 2 waves, in two LDS stages of
// 128 bytes of K: the pipeline of gemm_tile16.hpp, of which a k-step is two
// substeps of 64 bytes.
template <typename T, typename TOut, bool GATED, int BM, int BN>
__global__ __launch_bounds__(256) void tile_kernel(Args a) {
  constexpr int NW = 4, WM = BM / 2, WN = BN / 2, TM = WM / 16, TN = WN / 16, OUT = GATED ? BN / 2 : BN;
  constexpr int ES = sizeof(T);
  constexpr int A_BYTES = BM * kRowBytes, B_BYTES = BN * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char sA0[A_BYTES];
  __shared__ __attribute__((aligned(1024))) char sA1[A_BYTES];
  __shared__ __attribute__((aligned(1024))) char sB0[B_BYTES];
  __shared__ __attribute__((aligned(1024))) char sB1[B_BYTES];
  __shared__ int xrow[BM];
  __shared__ Edges<BM, BN> edges;
  struct Stage {
    char* a;
    char* b;
  };
  const Stage stage0{sA0, sB0}, stage1{sA1, sB1};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / 2, wn = wave % 2;
  const Found f = find_tile<BM, 4>(a, blockIdx.x, lane);
  if (f.group < 0) return;
  fill_edges<T, TOut, GATED>(a, f, edges, xrow, tid, 256);
  __syncthreads();

  const int row_bytes = a.K * ES, KT = max(2, (row_bytes + kRowBytes - 1) / kRowBytes), pad = KT * kRowBytes - row_bytes;
  const int64_t xpitch = a.ldx * ES, wpitch = a.ldw * ES;
  // X from its first row where rows are gathered, else from the tile's
  const int x0 = a.gather ? 0 : f.begin, n0 = f.tn * OUT;
  const RowLoader<BM, NW> la((const char*)a.X + x0 * xpitch, (a.gather ? a.rows / a.per : a.rows - x0) * xpitch, pad, tid,
                             [&](int r) __attribute__((always_inline)) {
                               return xrow[r] < 0 ? (int64_t)-1 : (xrow[r] - x0) * xpitch;
                             });
  const RowLoader<BN, NW> lb((const char*)a.W + f.group * a.group_w * ES + n0 * wpitch,
                             ((GATED ? 2 : 1) * (int64_t)a.N - n0) * wpitch, pad, tid,
                             [&](int r) __attribute__((always_inline)) {
                               const int n = column_of<GATED>(r);
                               return n0 + n < a.N ? (n + (GATED && (r & 16) ? (int64_t)a.N : 0)) * wpitch : (int64_t)-1;
                             });

  // Fragment rows w0 + 16 f + lane % 16 have the swizzle lane % 8: one offset
  // per operand and substep, the rest immediate.
  const int sl = lane & 7;
  int aoff[2], boff[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    aoff[kk] = (wm * WM + (lane & 15)) * kRowBytes + (((4 * kk + (lane >> 4)) ^ sl) << 4);
    boff[kk] = (wn * WN + (lane & 15)) * kRowBytes + (((4 * kk + (lane >> 4)) ^ sl) << 4);
  }
  typename Elem<T>::acc acc[TM][TN] = {};
  u32x4 fa[2][TM], fb[2][TN];
  auto read_frag = [&](const Stage& st, int kk, int f, u32x4 (&xa)[TM], u32x4 (&xb)[TN]) __attribute__((always_inline)) {
    if (f < TN) xb[f] = *(const u32x4*)(st.b + boff[kk] + f * 16 * kRowBytes);
    else xa[f - TN] = *(const u32x4*)(st.a + aoff[kk] + (f - TN) * 16 * kRowBytes);
  };
  constexpr int NMF = TM * TN, NDR = TM + TN, NDA = RowLoader<BM, NW>::NI, NDL = NDA + RowLoader<BN, NW>::NI;
  auto substep = [&](auto sub_c, const u32x4 (&xa)[TM], const u32x4 (&xb)[TN], const Stage& rd, int rd_kk, bool do_read,
                     u32x4 (&na)[TM], u32x4 (&nb)[TN], const Stage& to, bool do_copy, int kt) __attribute__((always_inline)) {
    constexpr int sub = decltype(sub_c)::value;
    static_for<NMF>([&](auto slot_c) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_c)::value, i = slot / TN, j = slot % TN;
      acc[i][j] = mfma<T>(xb[j], xa[i], acc[i][j]);
      static_for<NDR>([&](auto r_c) __attribute__((always_inline)) {
        constexpr int r = decltype(r_c)::value;
        if constexpr (r * NMF / NDR == slot)
          if (do_read) read_frag(rd, rd_kk, r, na, nb);
      });
      if constexpr (sub == 1) {
        if (do_copy) {
          static_for<NDL>([&](auto d_c) __attribute__((always_inline)) {
            constexpr int d = decltype(d_c)::value;
            if constexpr (d * NMF / NDL == slot) {
              if constexpr (d < NDA) la.issue(to.a, kt + 2, d);
              else lb.issue(to.b, kt + 2, d - NDA);
            }
          });
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto kstep = [&](const Stage& cur, const Stage& nxt, int kt, bool more1, bool more2) __attribute__((always_inline)) {
    substep(std::integral_constant<int, 0>{}, fa[0], fb[0], cur, 1, true, fa[1], fb[1], cur, false, kt);
    // this wave's copies of tile kt + 1 are its only outstanding ones
    tile::kloop_barrier<0>();
    __builtin_amdgcn_sched_barrier(0);
    substep(std::integral_constant<int, 1>{}, fa[1], fb[1], nxt, 0, more1, fa[0], fb[0], cur, more2, kt);
  };
  // Tile t lives in stage (t + KT) % 2: the last two k-steps are peeled.
  auto prologue = [&](const Stage& first, const Stage& second) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < NDL; ++d) {
      if (d < NDA) la.issue_first(first.a, 0, d, pad);
      else lb.issue_first(first.b, 0, d - NDA, pad);
    }
#pragma unroll
    for (int d = 0; d < NDL; ++d) {
      if (d < NDA) la.issue_first(second.a, 1, d, pad);
      else lb.issue_first(second.b, 1, d - NDA, pad);
    }
    tile::kloop_barrier<NDL>();
#pragma unroll
    for (int f = 0; f < NDR; ++f) read_frag(first, 0, f, fa[0], fb[0]);
  };
  int kt = 0;
  if (KT & 1) {
    prologue(stage1, stage0);
    kstep(stage1, stage0, 0, true, true);
    kt = 1;
  } else {
    prologue(stage0, stage1);
  }
  for (; kt + 4 <= KT; kt += 2) {
    kstep(stage0, stage1, kt, true, true);
    kstep(stage1, stage0, kt + 1, true, true);
  }
  kstep(stage0, stage1, kt, true, false);
  kstep(stage1, stage0, kt + 1, false, false);

  // Every wave is done with the stages: their memory stages the outputs.
  __syncthreads();
  static_assert(16 * WN * 2 <= A_BYTES && 16 * WN * 2 <= B_BYTES, "staging area");
  char* const mine = wave == 0 ? sA0 : wave == 1 ? sA1 : wave == 2 ? sB0 : sB1;
  with_activation(a.epi, [&](auto act) __attribute__((always_inline)) {
    write_rows<T, TOut, GATED, decltype(act)::value>(a, acc, edges, wm * WM, wn * WN, n0 + wn * (OUT / 2), lane, mine);
  });
}

// ---------------------------------------------------------------------------
// the streaming kernel, for few rows a group
// ---------------------------------------------------------------------------
// BM rows and 32 rows of W by four waves that share K: wave w takes every
// fourth piece of 128 bytes, through a ring of P slots of its own LDS, so that
// nothing but a wave's own loads is waited for; their sums are added at the
// end, in the waves' order.  The pieces begin apart for each workgroup: where
// all read the same places of rows a power of two apart, the memory's channels
// are used unevenly.  W passes the caches by where a group's rows are one tile.
template <typename T, typename TOut, bool GATED, int BM, int P>
__global__ __launch_bounds__(256, 2) void stream_kernel(Args a) {
  constexpr int BN = 32, NW = 4, TM = BM / 16, ES = sizeof(T), OUT = GATED ? 16 : 32;
  constexpr int SLOT = BN * kRowBytes;
  using Acc = typename Elem<T>::acc;
  __shared__ __attribute__((aligned(1024))) char slots[P][NW * SLOT];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Found f = find_tile<BM, 4>(a, blockIdx.x, lane);
  if (f.group < 0) return;
  const int row_bytes = a.K * ES, KT = (row_bytes + kRowBytes - 1) / kRowBytes, pad = KT * kRowBytes - row_bytes;
  const int64_t xpitch = a.ldx * ES, wpitch = a.ldw * ES;
  const int n0 = f.tn * OUT;
  // (one wave's instructions: 8 rows each)
  const RowLoader<BN, 1> lb((const char*)a.W + f.group * a.group_w * ES + n0 * wpitch,
                            ((GATED ? 2 : 1) * (int64_t)a.N - n0) * wpitch, pad, lane,
                            [&](int r) __attribute__((always_inline)) {
                              const int n = column_of<GATED>(r);
                              return n0 + n < a.N ? (n + (GATED && (r & 16) ? (int64_t)a.N : 0)) * wpitch : (int64_t)-1;
                            });
  // this lane's rows of X, as operands
  const int x0 = a.gather ? 0 : f.begin;
  const __amdgpu_buffer_rsrc_t xr = tile::make_rsrc(
      (const char*)a.X + x0 * xpitch - pad,
      (uint32_t)min((a.gather ? a.rows / a.per : a.rows - x0) * xpitch + pad, (int64_t)0xfffff000));
  int entry[TM];
  uint32_t xoff[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int at = f.begin + 16 * i + c;
    entry[i] = at < f.end ? entry_of(a, at) : -1;
    const int row = a.gather ? entry[i] / a.per : at;
    // (none: past the buffer's end with a piece's second half added too)
    xoff[i] = entry[i] < 0 ? 0xFFFFFF00u : (uint32_t)((row - x0) * xpitch) + 16 * h;
  }

  const int n = wave < KT ? (KT - wave + NW - 1) / NW : 0;  // this wave's pieces
  int next = n > 0 ? blockIdx.x % n : 0, left = n;
  char* const ring = &slots[0][0];
  u32x4 x[P][TM][2];
  auto issue = [&](auto slot_c) __attribute__((always_inline)) {
    constexpr int J = decltype(slot_c)::value;
    // (past the last piece: zeros, no access)
    const int kt = left <= 0 ? 0 : next * NW + wave, pad0 = left <= 0 ? 1 << 30 : kt == 0 ? pad : 0;
    --left;
    if (++next >= n) next = 0;
#pragma unroll
    for (int i = 0; i < BN / 8; ++i) {
      const uint32_t v = 16 * lb.chunk < pad0 ? 0xFFFFFFF0u : lb.voff[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(lb.rsrc, (lds_ptr)(slots[J] + wave * SLOT + i * 1024), 16, v, kt * kRowBytes, 0, 2);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        x[J][i][kk] = tile::load16(xr, 64 * kk + 16 * h < pad0 ? 0xFFFFFFF0u : xoff[i] + 64 * kk, kt * kRowBytes);
  };
  Acc acc[TM][2] = {};
  auto multiply = [&](auto slot_c) __attribute__((always_inline)) {
    constexpr int J = decltype(slot_c)::value;
    const char* s = slots[J] + wave * SLOT;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 w = *(const u32x4*)(s + (16 * j + c) * kRowBytes + (((4 * kk + h) ^ (c & 7)) << 4));
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[i][j] = mfma<T>(w, x[J][i][kk], acc[i][j]);
      }
  };
  constexpr int OPS = BN / 8 + 2 * TM;
  static_for<P - 1>([&](auto j) __attribute__((always_inline)) { issue(j); });
  for (int i = 0; i < n; i += P)
    static_for<P>([&](auto j) __attribute__((always_inline)) {
      issue(std::integral_constant<int, (decltype(j)::value + P - 1) % P>{});
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((P - 1) * OPS));
      asm volatile("" ::: "memory");
      multiply(j);
    });

  // The waves' sums, four columns of a row a thread, in the ring's memory, once
  // the zeros past the last pieces have been written there.
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  __syncthreads();
  Acc* const red = (Acc*)ring;
  static_assert(NW * TM * 2 * 64 * 16 <= NW * SLOT * P, "the sums fit the ring");
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) red[(wave * TM * 2 + 2 * i + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  constexpr int ITEMS = TM * (GATED ? 1 : 2);  // of 64 threads each
  if (wave >= ITEMS) return;
  const int i = GATED ? wave : wave >> 1, j = GATED ? 0 : wave & 1;
  const int row = f.begin + 16 * i + c, q = row < f.end ? entry_of(a, row) : -1;
  if (q < 0) return;
  const int col = n0 + 16 * j + 4 * h;
  const int64_t g0 = (int64_t)f.group * a.N * (GATED ? 2 : 1) + col;
  const bool biased = has_bias(a.epi);
  const float xs = Elem<T>::kInt ? a.xs[a.gather ? q / a.per : row] : 1.0f;
  auto z = [&](int jj, int64_t at) __attribute__((always_inline)) {
    Acc s = red[(2 * i + jj) * 64 + lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += red[(w * TM * 2 + 2 * i + jj) * 64 + lane];
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = (float)s[e];
      if (col + e >= a.N) continue;
      if constexpr (Elem<T>::kInt) v[e] = v[e] * xs * a.ws[at + e];
      if (biased) v[e] += to_f32(((const TOut*)a.bias)[at + e]);
    }
    return v;
  };
  const int to = a.scatter ? q : row;
  with_activation(a.epi, [&](auto act) __attribute__((always_inline)) {
    f32x4 v = z(j, g0);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activated<decltype(act)::value>(v[e]);
    if constexpr (GATED) v *= z(1, g0 + a.N);
    TOut* out = (TOut*)a.C + to * a.ldc + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e >= a.N) continue;
      if (!GATED && a.R) v[e] += to_f32(((const TOut*)a.R)[to * a.ldr + col + e]);
      out[e] = from_f32<TOut>(v[e]);
    }
  });
}

template <typename T, typename TOut, int BM, int BN>
hipError_t launch_tiles(Args a, bool gated, hipStream_t stream) {
  const int cols = gated ? BN / 2 : BN;
  a.tiles_n = (a.N + cols - 1) / cols;
  // tiles of rows of all groups: what their ends can add
  const int64_t tiles_m = a.offsets ? a.rows / BM + std::min(a.groups, a.rows) : (a.rows + BM - 1) / BM;
  const dim3 grid((uint32_t)(tiles_m * a.tiles_n)), block(256);
  if (gated) hipLaunchKernelGGL((tile_kernel<T, TOut, true, BM, BN>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((tile_kernel<T, TOut, false, BM, BN>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <typename T, typename TOut, int BM, int P>
hipError_t launch_stream(Args a, bool gated, hipStream_t stream) {
  const int cols = gated ? 16 : 32;
  a.tiles_n = (a.N + cols - 1) / cols;
  const int64_t tiles_m = a.offsets ? a.rows / BM + std::min(a.groups, a.rows) : (a.rows + BM - 1) / BM;
  const dim3 grid((uint32_t)(tiles_m * a.tiles_n)), block(256);
  if (gated) hipLaunchKernelGGL((stream_kernel<T, TOut, true, BM, P>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((stream_kernel<T, TOut, false, BM, P>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <typename T, typename TOut>
hipError_t launch(Args a, bool gated, hipStream_t stream) {
  if (a.rows <= 16 * a.groups) return launch_stream<T, TOut, 16, 4>(a, gated, stream);
  if (a.rows <= 32 * a.groups) return launch_stream<T, TOut, 32, 4>(a, gated, stream);
  if (a.rows >= 128 * a.groups) return launch_tiles<T, TOut, 256, 256>(a, gated, stream);
  const int cols = gated ? 32 : 64;
  a.tiles_n = (a.N + cols - 1) / cols;
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
