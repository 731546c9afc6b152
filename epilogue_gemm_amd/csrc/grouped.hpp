// grouped.hpp -- products of rows with the weights of their groups,
//
//     C[.] = act(X[.] W[g]^T + bias[g])   or   act(gate) * up
//
// for 16-bit formats and, with scales, 8-bit integers; one group of all rows
// is the 8-bit product.  Two kernels on v_mfma_f32_16x16x32 and its 8-bit like
// v_mfma_i32_16x16x64_i8, whose operands are the same 16 bytes a lane, so that one
// layout in LDS serves both:
//   * tile_kernel: tiles of 64 x 64 to 256 x 256, rows of X gathered by the direct
//     copies themselves, the group found by each workgroup from the offsets.  Large
//     ones are bound by the power limit (i8 8192^3 398 to 440 us, 2.5 to 2.8 POP/s;
//     under counters 467 us at 1.77 GHz of 2.4 with the matrix units 67 % busy;
//     bf16, 8 groups of 16384 rows, 2 x 4096 of 4096, 860 to 900 us, 1.22 to 1.28
//     PFLOP/s, 925 us at 1.78 GHz, 72 %), those of short K by the epilogue and the
//     lookups (32 groups of 12284 rows, 4096 of 2048, i8: 159 to 164 us, of which the
//     matrix units are busy 41 %), small ones by the latency of a k-step (1001 x 2055
//     x 4096, i8: 21 to 22 us for 32 of them, 21 % busy);
//   * stream_kernel: for few rows a group, bound by W from HBM (32 tokens, 4 of 64,
//     2 x 1024 of 2048, bf16: 80.0 us, 6.0 TB/s, 1.00 x the least bytes).
// Measured and not kept: a workgroup a tile of the streaming kernel (83.9 us for
// 80.5), twice its ring with one workgroup a CU (82.8), 32 or 64 rows a tile there
// (X as operands for rows that mostly are none: 88.7, 105); 128 x 256 tiles of three
// stages (531 us for 398 at 8192^3); 64 x 64 with eight stages, a workgroup a CU
// (i8, 64 x 2048 x 8192 13.5 us for 13.5, 32 rows 12.1 for 12.9; 1024 x 2560 x 4096
// 24.4 for 20.0, 2048 x 4096 x 4096 65 for 52); the epilogue's
// bands staged apart, each stored while the next one is formed (164 us for 160
// in 12284 rows of 32 groups).
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

// (an access off its alignment is one instruction all the same)
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

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

// Offset g, of those that may hold anything.
__device__ __forceinline__ int clamped(const Args& a, int g) { return max(0, min(a.offsets[g], a.rows)); }

// Offsets that descend somewhere count as no lower than any before them, so that
// no place is of two groups and a grid for ascending ones holds all tiles.  The
// group that has tile f (-1: none) and its places [begin, end), by a walk from the
// first group on; f is then the tile's number in the group, of `tiles` of rows.
template <int BM>
__device__ __forceinline__ int walk_raised(const Args& a, uint32_t& f, int& begin, int& end, int& tiles) {
  end = clamped(a, 0);
  for (int g = 0; g < a.groups; ++g) {
    begin = end;
    end = max(begin, clamped(a, g + 1));
    tiles = (end - begin + BM - 1) / BM;
    const uint32_t all = (uint32_t)tiles * (uint32_t)a.tiles_n;
    if (f < all) return g;
    f -= all;
  }
  return -1;
}

// A tile of those of all groups, from the workgroup's number.  Workgroups go to
// the 8 XCDs in turn: consecutive tiles go to one XCD, group by group, in each
// in panels of PANEL tiles of rows, column by column, so that the tiles which
// one XCD works on together share rows of X and of W in its L2.  Every wave
// counts the tiles of the groups for itself, lane l those of groups l * per ..
// + per - 1.
template <int BM, int PANEL>
__device__ __forceinline__ Found find_tile(const Args& a, int id, int lane) {
  int own = 0, g0 = 0, g1 = 0, incl = 0, total;
  bool descends = false;
  if (a.offsets) {
    const int per = (a.groups + 63) / 64;
    g0 = min(lane * per, a.groups);
    g1 = min(g0 + per, a.groups);
    int signs = 0;
    for (int g = g0; g < g1; ++g) {
      const int n = clamped(a, g + 1) - clamped(a, g);
      own += (max(0, n) + BM - 1) / BM;
      signs |= n;
    }
    descends = __builtin_amdgcn_ballot_w64(signs < 0) != 0;
    incl = wave::scan(own);
    total = __builtin_amdgcn_readlane(incl, 63);
  } else {
    total = (a.rows + BM - 1) / BM;
  }
  const uint32_t all = (uint32_t)total * (uint32_t)a.tiles_n;
  if (!descends && (uint32_t)id >= all) return Found{-1, 0, 0, 0};
  const uint32_t x = id & 7, f = x * (all >> 3) + min(x, all & 7) + ((uint32_t)id >> 3);
  int g = 0, begin = 0, end = a.rows, tiles = total, at = (int)f;
  if (__builtin_expect(descends, 0)) {
    uint32_t left = (uint32_t)id;
    g = walk_raised<BM>(a, left, begin, end, tiles);
    if (g < 0) return Found{-1, 0, 0, 0};
    at = (int)left;
  } else if (a.offsets) {
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
template <int R, int NW, int AUX = 0>
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
                                             kt * kRowBytes, 0, AUX);
  }
  __device__ __forceinline__ void issue_first(char* dst, int kt, int i, int pad) const {
    const uint32_t v = 16 * chunk + kt * kRowBytes < pad ? 0xFFFFFFF0u : voff[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(dst + (NW * i + wave) * 1024), 16, v, kt * kRowBytes, 0, AUX);
  }
};

// What the epilogue needs of a tile's rows and columns, in LDS.
template <int BM, int BN>
struct Edges {
  int c[BM];      // row of C, -1: none
  float xs[BM];   // a row's scale (8-bit rows)
  f32x4 ws[BN / 4], bias[BN / 4];  // of each row of the tile of W
};

// By 256 threads, thread r with the entry q of row r (-1: none).  The tile's rows
// of X, -1 for none, are left in xrow.
template <typename T, typename TOut, bool GATED, int BM, int BN>
__device__ __forceinline__ void fill_edges(const Args& a, const Found& f, Edges<BM, BN>& edges, int* xrow, int tid, int q) {
  static_assert(BM <= 256 && BN <= 256, "a thread a row");
  if (tid < BM) {
    const int i = f.begin + tid, x = q < 0 ? -1 : a.gather ? q / a.per : i;
    xrow[tid] = x;
    edges.c[tid] = q < 0 ? -1 : a.scatter ? q : i;
    if constexpr (Elem<T>::kInt) edges.xs[tid] = q < 0 ? 0.0f : a.xs[x];
  }
  const bool biased = has_bias(a.epi);
  if (const int r = tid; r < BN) {
    const int n = f.tn * (GATED ? BN / 2 : BN) + column_of<GATED>(r);
    const int64_t at = (int64_t)f.group * a.N * (GATED ? 2 : 1) + (GATED && (r & 16) ? a.N : 0) + n;
    if constexpr (Elem<T>::kInt) ((float*)edges.ws)[r] = n < a.N ? a.ws[at] : 0.0f;
    ((float*)edges.bias)[r] = biased && n < a.N ? to_f32(((const TOut*)a.bias)[at]) : 0.0f;
  }
}

// Four values of a row of the residual, those past the last column zeros.
template <typename TOut>
__device__ __forceinline__ u32x2 residual4(const TOut* r, int n, int N) {
  if (n + 4 <= N) return *(const u32x2_any*)r;
  u32x2 w = {};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < N) w[e >> 1] |= (uint32_t)bits16(r[e]) << (16 * (e & 1));
  return w;
}

// Epilogue of a wave's TM x TN blocks of 16 x 16 (lane (c, h) has columns 4 h
// .. + 3 of row c of each), rows r0 .. and W's rows w0 .. of the tile, output
// columns n0 ..: the scales, bias, activation, gate's product or residual in
// fp32, one rounding, then each band of 16 rows through the wave's own LDS
// (16-byte chunks swizzled by row) and out in 16-byte pieces along rows.  What
// belongs to columns is read once, a band's residual while the band before it
// is worked on.
template <typename T, typename TOut, bool GATED, int ACT, bool RES, int TM, int TN, int BM, int BN>
__device__ __forceinline__ void write_rows(const Args& a, const typename Elem<T>::acc (&acc)[TM][TN],
                                           const Edges<BM, BN>& edges, int r0, int w0, int n0, int lane, char* stage) {
  constexpr int W = (GATED ? TN / 2 : TN) * 16;   // output columns
  constexpr int CPR = W * 2 / 16, SWM = (CPR < 16 ? CPR : 16) - 1, RPI = 64 / CPR < 16 ? 64 / CPR : 16;
  constexpr int S = GATED ? 2 : 1;
  const int c = lane & 15, h = lane >> 4;
  f32x4 ws[Elem<T>::kInt ? TN : 1], bias[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    if constexpr (Elem<T>::kInt) ws[j] = edges.ws[w0 / 4 + 4 * j + h];
    bias[j] = edges.bias[w0 / 4 + 4 * j + h];
  }
  u32x2 res[RES ? 2 : 1][RES ? TN : 1];
  auto load_residual = [&](int i, u32x2 (&r)[RES ? TN : 1]) __attribute__((always_inline)) {
    const int to = edges.c[r0 + 16 * i + c];
    if (to < 0) return;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + 16 * j + 4 * h;
      r[j] = residual4((const TOut*)a.R + to * a.ldr + n, n, a.N);
    }
  };
  if constexpr (RES) load_residual(0, res[0]);
  static_for<TM>([&](auto i_c) __attribute__((always_inline)) {
    constexpr int i = decltype(i_c)::value;
    const int row = r0 + 16 * i;
    const float xs = Elem<T>::kInt ? edges.xs[row + c] : 1.0f;
    if constexpr (RES && i + 1 < TM) load_residual(i + 1, res[(i + 1) & 1]);
    static_for<TN / S>([&](auto j_c) __attribute__((always_inline)) {
      constexpr int j = decltype(j_c)::value;
      auto z = [&](auto jj_c) __attribute__((always_inline)) {
        constexpr int jj = decltype(jj_c)::value;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][jj][e];
        if constexpr (Elem<T>::kInt) v = v * xs * ws[jj];
        return v + bias[jj];
      };
      f32x4 v = z(std::integral_constant<int, S * j>{});
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = activated<ACT>(v[e]);
      if constexpr (GATED) v *= z(std::integral_constant<int, 2 * j + 1>{});
      if constexpr (RES) {
        const u32x2 w = res[i & 1][j];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += to_f32(__builtin_bit_cast(TOut, (uint16_t)(w[e >> 1] >> (16 * (e & 1)))));
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
      const char* src = stage + r * (W * 2) + ((ch ^ (r & SWM)) << 4);
      const int cr = edges.c[row + r], n = n0 + 8 * ch;
      if (cr < 0 || n >= a.N) continue;
      uint16_t* dst = (uint16_t*)a.C + cr * a.ldc + n;
      if (n + 8 <= a.N) {
        *(u32x4_any*)dst = *(const u32x4*)src;
      } else {
#pragma unroll 1
        for (int e = 0; e < a.N - n; ++e) dst[e] = ((const uint16_t*)src)[e];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Stage J of a ring: an object of its own, so that the compiler can tell a read
// of one stage from a copy in flight into another (of one array of all stages,
// it waits for every copy before a read: 229 us for 184).
template <int J, int BYTES>
__device__ __forceinline__ char* ring_stage() {
  __shared__ __attribute__((aligned(1024))) char stage[BYTES];
  return stage;
}

// BM x BN products (BN / 2 gated outputs) of tile f by WGM x 4 / WGM waves, in
// a ring of P LDS stages (of STAGE bytes) of 128 bytes of K: the pipeline of
// gemm_tile16.hpp, of which a k-step is two substeps of 64 bytes:
//   substep 0   multiply the first half of tile kt, read its second;
//   barrier     after this wave's copies of tile kt + 1 have landed: every wave
//               is done reading tile kt's stage, tile kt + 1 is whole;
//   substep 1   multiply the second half, read the first of tile kt + 1, and
//               copy tile kt + P into the stage that tile kt leaves.
template <typename T, typename TOut, bool GATED, int BM, int BN, int P, bool PAST, int WGM, int STAGE, int EM>
__device__ __forceinline__ void multiply_tile(const Args& a, const Found& f, Edges<EM, BN>& edges, int* xrow, int tid) {
  constexpr int NW = 4, WGN = NW / WGM, WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16, OUT = GATED ? BN / 2 : BN;
  constexpr int ES = sizeof(T);
  constexpr int A_BYTES = BM * kRowBytes, B_BYTES = BN * kRowBytes;
  static_assert(A_BYTES + B_BYTES <= STAGE && BM <= EM, "the stage holds the tile");
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN;

  // (the first k-steps hold what is missing to a multiple of P)
  const int row_bytes = a.K * ES, rounds = (row_bytes + P * kRowBytes - 1) / (P * kRowBytes);
  const int pad = rounds * P * kRowBytes - row_bytes;
  const int64_t xpitch = a.ldx * ES, wpitch = a.ldw * ES;
  constexpr int NDA = RowLoader<BM, NW>::NI, NDB = RowLoader<BN, NW>::NI, NDL = NDA + NDB;
  const int q = tid < BM && f.begin + tid < f.end ? entry_of(a, f.begin + tid) : -1;
  const int n0 = f.tn * OUT;
  const RowLoader<BN, NW, PAST ? 2 : 0> lb((const char*)a.W + f.group * a.group_w * ES + n0 * wpitch,
                             ((GATED ? 2 : 1) * (int64_t)a.N - n0) * wpitch, pad, tid,
                             [&](int r) __attribute__((always_inline)) {
                               const int n = column_of<GATED>(r);
                               return n0 + n < a.N ? (n + (GATED && (r & 16) ? (int64_t)a.N : 0)) * wpitch : (int64_t)-1;
                             });
  auto first_b = [&](auto j) __attribute__((always_inline)) {
    constexpr int J = decltype(j)::value;
#pragma unroll
    for (int d = 0; d < NDB; ++d) lb.issue_first(ring_stage<J, STAGE>() + A_BYTES, J, d, pad);
  };
  // With two stages W's first copies are on their way while the rows of X are
  // looked up (with more, the loop's waits count copies tile by tile).
  if constexpr (P == 2) static_for<P>(first_b);
  fill_edges<T, TOut, GATED>(a, f, edges, xrow, tid, q);
  __syncthreads();
  // X from its first row where rows are gathered, else from the tile's
  const int x0 = a.gather ? 0 : f.begin;
  const RowLoader<BM, NW> la((const char*)a.X + x0 * xpitch, (a.gather ? a.rows / a.per : a.rows - x0) * xpitch, pad, tid,
                             [&](int r) __attribute__((always_inline)) {
                               return xrow[r] < 0 ? (int64_t)-1 : (xrow[r] - x0) * xpitch;
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
  auto read_frag = [&](auto slot_c, int kk, int f, u32x4 (&xa)[TM], u32x4 (&xb)[TN]) __attribute__((always_inline)) {
    constexpr int S = decltype(slot_c)::value;
    char* const st = ring_stage<S, STAGE>();
    if (f < TN) xb[f] = *(const u32x4*)(st + A_BYTES + boff[kk] + f * 16 * kRowBytes);
    else xa[f - TN] = *(const u32x4*)(st + aoff[kk] + (f - TN) * 16 * kRowBytes);
  };
  constexpr int NMF = TM * TN, NDR = TM + TN;
  // NMF slots of one product and its share of the reads and copies; nothing
  // moves across a slot's end.
  auto substep = [&](auto sub_c, const u32x4 (&xa)[TM], const u32x4 (&xb)[TN], auto rd, int rd_kk, auto do_read,
                     u32x4 (&na)[TM], u32x4 (&nb)[TN], auto to, auto do_copy, int kt) __attribute__((always_inline)) {
    constexpr int sub = decltype(sub_c)::value, S = decltype(to)::value;
    static_for<NMF>([&](auto slot_c) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_c)::value, i = slot / TN, j = slot % TN;
      acc[i][j] = mfma<T>(xb[j], xa[i], acc[i][j]);
      if constexpr (decltype(do_read)::value) {
        static_for<NDR>([&](auto r_c) __attribute__((always_inline)) {
          constexpr int r = decltype(r_c)::value;
          if constexpr (r * NMF / NDR == slot) read_frag(rd, rd_kk, r, na, nb);
        });
      }
      if constexpr (sub == 1 && decltype(do_copy)::value) {
        static_for<NDL>([&](auto d_c) __attribute__((always_inline)) {
          constexpr int d = decltype(d_c)::value;
          if constexpr (d * NMF / NDL == slot) {
            char* const st = ring_stage<S, STAGE>();
            if constexpr (d < NDA) la.issue(st, kt + P, d);
            else lb.issue(st + A_BYTES, kt + P, d - NDA);
          }
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // k-step kt = P round + J; the last round copies nothing more
  auto kstep = [&](auto slot_c, auto last_c, int kt) __attribute__((always_inline)) {
    constexpr int J = decltype(slot_c)::value;
    constexpr bool LAST = decltype(last_c)::value;
    constexpr std::integral_constant<int, J> cur{};
    constexpr std::integral_constant<int, (J + 1) % P> nxt{};
    substep(std::integral_constant<int, 0>{}, fa[0], fb[0], cur, 1, std::true_type{}, fa[1], fb[1], cur, std::false_type{}, kt);
    // copies of tile kt + 2 and on may be outstanding
    tile::kloop_barrier<NDL * (LAST ? (P - 2 - J > 0 ? P - 2 - J : 0) : P - 2)>();
    __builtin_amdgcn_sched_barrier(0);
    substep(std::integral_constant<int, 1>{}, fa[1], fb[1], nxt, 0, std::bool_constant<!(LAST && J == P - 1)>{}, fa[0], fb[0],
            cur, std::bool_constant<!LAST>{}, kt);
  };
  static_for<P>([&](auto j) __attribute__((always_inline)) {
    constexpr int J = decltype(j)::value;
#pragma unroll
    for (int d = 0; d < NDA; ++d) la.issue_first(ring_stage<J, STAGE>(), J, d, pad);
    if constexpr (P > 2) first_b(j);
  });
  tile::kloop_barrier<(P == 2 ? NDA : NDL * (P - 1))>();
#pragma unroll
  for (int f = 0; f < NDR; ++f) read_frag(std::integral_constant<int, 0>{}, 0, f, fa[0], fb[0]);
  int kt = 0;
  // (128 accumulators a lane and more: without a round before the loop they are copied
  // between register files around every product)
  if constexpr (NMF == 64 || WGM == 1) {
    if (rounds > 1) {
      static_for<P>([&](auto j) __attribute__((always_inline)) { kstep(j, std::false_type{}, decltype(j)::value); });
      kt = P;
    }
  }
  for (; kt < (rounds - 1) * P; kt += P)
    static_for<P>([&](auto j) __attribute__((always_inline)) { kstep(j, std::false_type{}, kt + decltype(j)::value); });
  static_for<P>([&](auto j) __attribute__((always_inline)) { kstep(j, std::true_type{}, kt + decltype(j)::value); });

  // Every wave is done with the stages: their memory stages the outputs.
  __syncthreads();
  static_assert(NW * 16 * WN * 2 <= A_BYTES + B_BYTES, "staging area");
  char* const mine = ring_stage<0, STAGE>() + wave * (16 * WN * 2);
  with_activation(a.epi, [&](auto act) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act)::value;
    const int n = n0 + wn * (OUT / WGN);
    if constexpr (Elem<T>::kInt && !GATED) {
      if (a.R) {
        write_rows<T, TOut, GATED, ACT, true>(a, acc, edges, wm * WM, wn * WN, n, lane, mine);
        return;
      }
    }
    write_rows<T, TOut, GATED, ACT, false>(a, acc, edges, wm * WM, wn * WN, n, lane, mine);
  });
}

// A tile a workgroup.  Of 256 rows (P = 2), those of at most 128 are done by waves
// beside each other, in half the products.
template <typename T, typename TOut, bool GATED, int BM, int BN, int P, bool PAST>
__global__ __launch_bounds__(256) void tile_kernel(Args a) {
  constexpr int STAGE = (BM + BN) * kRowBytes;
  __shared__ int xrow[BM];
  __shared__ Edges<BM, BN> edges;
  const int tid = threadIdx.x;
  const Found f = find_tile<BM, 4>(a, blockIdx.x, tid & 63);
  if (f.group < 0) return;
  if constexpr (BM == 256) {
    if (f.end - f.begin <= 128) {
      multiply_tile<T, TOut, GATED, 128, BN, P, PAST, 1, STAGE>(a, f, edges, xrow, tid);
      return;
    }
  }
  multiply_tile<T, TOut, GATED, BM, BN, P, PAST, 2, STAGE>(a, f, edges, xrow, tid);
}

// ---------------------------------------------------------------------------
// the streaming kernel, for few rows a group
// ---------------------------------------------------------------------------
// A tile and its way to the next one: within a group the tiles of rows first,
// then columns.
template <int BM>
struct Walk {
  int group, begin, end;  // places of the group
  int tiles, m, tn;       // tiles of its rows; this one
  // `group`, the one before it ending at `end`
  __device__ __forceinline__ void enter(const Args& a) {
    begin = end;
    end = a.offsets ? max(begin, clamped(a, group + 1)) : a.rows;
    tiles = (end - begin + BM - 1) / BM;
  }
  // true: to other rows.  (There is a next tile, or this one stays.)
  __device__ __forceinline__ bool next(const Args& a) {
    if (++m < tiles) return true;
    m = 0;
    if (++tn < a.tiles_n) return tiles > 1;
    tn = 0;
    do {
      if (++group >= a.groups) {
        tiles = 0;
        group = a.groups - 1;
        return false;
      }
      enter(a);
    } while (tiles == 0);
    return true;
  }
  __device__ __forceinline__ int row0() const { return begin + m * BM; }
};

// Tiles of all groups, and which one is number f of them: lane l counts those
// of groups l * per .. + per - 1, as find_tile does.
struct Count {
  int g0, g1, own, incl, total;
  bool descends;
};
template <int BM>
__device__ __forceinline__ Count count_tiles(const Args& a, int lane) {
  Count c{};
  if (!a.offsets) {
    c.total = (a.rows + BM - 1) / BM;
    return c;
  }
  const int per = (a.groups + 63) / 64;
  c.g0 = min(lane * per, a.groups);
  c.g1 = min(c.g0 + per, a.groups);
  int signs = 0;
  for (int g = c.g0; g < c.g1; ++g) {
    const int n = clamped(a, g + 1) - clamped(a, g);
    c.own += (max(0, n) + BM - 1) / BM;
    signs |= n;
  }
  c.descends = __builtin_amdgcn_ballot_w64(signs < 0) != 0;
  if (__builtin_expect(c.descends, 0)) {
    // (no tile has this number: the walk takes from it all that there are)
    uint32_t f = ~0u;
    int begin, end, tiles;
    walk_raised<BM>(a, f, begin, end, tiles);
    c.total = (int)(~f / (uint32_t)a.tiles_n);
    return c;
  }
  c.incl = wave::scan(c.own);
  c.total = __builtin_amdgcn_readlane(c.incl, 63);
  return c;
}
template <int BM>
__device__ __forceinline__ Walk<BM> walk_from(const Args& a, const Count& c, uint32_t f) {
  Walk<BM> w{};
  int at = (int)f;
  if (__builtin_expect(c.descends, 0)) {
    w.group = walk_raised<BM>(a, f, w.begin, w.end, w.tiles);
    w.tn = (int)f / w.tiles;
    w.m = (int)f - w.tn * w.tiles;
    return w;
  }
  if (a.offsets) {
    const uint32_t left = f - (uint32_t)(c.incl - c.own) * (uint32_t)a.tiles_n;
    const uint64_t owner = __builtin_amdgcn_ballot_w64(left < (uint32_t)c.own * (uint32_t)a.tiles_n);
    int g = c.g0;
    at = (int)left;
    for (; g < c.g1; ++g) {
      const int tiles = (max(0, clamped(a, g + 1) - clamped(a, g)) + BM - 1) / BM;
      if (at < tiles * a.tiles_n) break;
      at -= tiles * a.tiles_n;
    }
    const int src = __builtin_ctzll(owner);
    w.group = __builtin_amdgcn_readlane(g, src);
    at = __builtin_amdgcn_readlane(at, src);
    w.end = clamped(a, w.group);
  }
  w.enter(a);
  w.tn = at / w.tiles;
  w.m = at - w.tn * w.tiles;
  return w;
}

// Tiles of BM rows and 32 rows of W, shared out evenly over workgroups that stay:
// one stream of loads each, which runs on from tile to tile.  The four waves
// share K: wave w takes every fourth piece of 128 bytes, W's through a ring of P
// slots of its own LDS and X's as operands, so that a wave waits for its own
// loads alone; at a tile's end their sums are added in the waves' order.  The
// pieces begin apart for each workgroup: where all read the same places of rows
// a power of two apart, the memory's channels are used unevenly.
template <typename T, typename TOut, bool GATED, int BM, int P, bool PAST>
__global__ __launch_bounds__(256) void stream_kernel(Args a) {
  constexpr int BN = 32, NW = 4, TM = BM / 16, ES = sizeof(T), OUT = GATED ? 16 : 32;
  constexpr int SLOT = BN * kRowBytes;
  using Acc = typename Elem<T>::acc;
  __shared__ __attribute__((aligned(1024))) char slots[P][NW * SLOT];
  __shared__ Acc sums[2][NW][TM * 2][64];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Count count = count_tiles<BM>(a, lane);
  const uint32_t all = (uint32_t)count.total * (uint32_t)a.tiles_n, n = gridDim.x;
  // consecutive shares go to one XCD
  const uint32_t share = n % 8 == 0 ? blockIdx.x % 8 * (n / 8) + blockIdx.x / 8 : blockIdx.x;
  const uint32_t f0 = (uint32_t)((uint64_t)all * share / n), f1 = (uint32_t)((uint64_t)all * (share + 1) / n);
  if (f0 == f1) return;
  Walk<BM> ahead = walk_from<BM>(a, count, f0), now = ahead;
  if (now.tiles == 0) return;

  const int row_bytes = a.K * ES, KT = (row_bytes + kRowBytes - 1) / kRowBytes, pad = KT * kRowBytes - row_bytes;
  const int64_t xpitch = a.ldx * ES, wpitch = a.ldw * ES;
  const int pieces = (KT + NW - 1) / NW;  // of each wave, the last perhaps none

  // Where the loads are: a tile, and the pieces of it that are left.
  const int wc = (lane & 7) ^ (lane >> 3);  // this lane's chunk of W's rows
  __amdgpu_buffer_rsrc_t wr, xr;
  uint32_t woff[4], xoff[TM];
  int entry[TM];
  int left = pieces, place = blockIdx.x % pieces, tiles_left = (int)(f1 - f0);
  auto enter_rows = [&]() __attribute__((always_inline)) {
    const int r0 = ahead.row0(), x0 = a.gather ? 0 : r0;
    xr = tile::make_rsrc((const char*)a.X + x0 * xpitch - pad,
                         (uint32_t)min((a.gather ? a.rows / a.per : a.rows - x0) * xpitch + pad, (int64_t)0xfffff000));
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int at = r0 + 16 * i + c;
      entry[i] = at < ahead.end ? entry_of(a, at) : -1;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = a.gather ? entry[i] / a.per : r0 + 16 * i + c;
      // (none: past the buffer's end with a piece's second half added too)
      xoff[i] = entry[i] < 0 ? 0xFFFFFF00u : (uint32_t)((row - x0) * xpitch) + 16 * h;
    }
  };
  auto enter_columns = [&]() __attribute__((always_inline)) {
    const int n0 = ahead.tn * OUT;
    wr = tile::make_rsrc((const char*)a.W + ahead.group * a.group_w * ES + n0 * wpitch - pad,
                         (uint32_t)min(((GATED ? 2 : 1) * (int64_t)a.N - n0) * wpitch + pad, (int64_t)0xfffff000));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 3), k = column_of<GATED>(r);
      woff[i] = n0 + k < a.N ? (uint32_t)((k + (GATED && (r & 16) ? (int64_t)a.N : 0)) * wpitch) + 16 * wc : 0xFFFFFFF0u;
    }
  };
  enter_rows();
  enter_columns();
  u32x4 x[P][TM][2];
  auto issue = [&](auto slot_c) __attribute__((always_inline)) {
    constexpr int J = decltype(slot_c)::value;
    // (past the last piece: zeros, no access)
    const bool none = place * NW + wave >= KT || tiles_left <= 0;
    const int kt = none ? 0 : place * NW + wave, pad0 = none ? 1 << 30 : kt == 0 ? pad : 0;
#pragma unroll
    for (int i = 0; i < BN / 8; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_ptr)(slots[J] + wave * SLOT + i * 1024), 16,
                                               16 * wc < pad0 ? 0xFFFFFFF0u : woff[i], kt * kRowBytes, 0, PAST ? 2 : 0);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        x[J][i][kk] = tile::load16(xr, 64 * kk + 16 * h < pad0 ? 0xFFFFFF00u : xoff[i] + 64 * kk, kt * kRowBytes);
    if (++place == pieces) place = 0;
    if (--left == 0) {
      left = pieces;
      if (--tiles_left > 0) {
        if (ahead.next(a)) enter_rows();
        if (ahead.tiles == 0) tiles_left = 0;
        enter_columns();
      }
    }
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
  // The tile's outputs, four columns of a row a thread; alternate tiles have
  // alternate sums, so that one barrier a tile is enough.
  int parity = 0;
  auto write = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sums[parity][wave][2 * i + j][lane] = acc[i][j];
        acc[i][j] = Acc{};
      }
    tile::kloop_barrier<63>();  // (the loads go on)
    constexpr int ITEMS = TM * (GATED ? 1 : 2);  // of 64 threads each
    for (int item = wave; item < ITEMS; item += NW) {
      const int i = GATED ? item : item >> 1, j = GATED ? 0 : item & 1;
      const int row = now.row0() + 16 * i + c, q = row < now.end ? entry_of(a, row) : -1;
      if (q < 0) continue;
      const int col = now.tn * OUT + 16 * j + 4 * h;
      const int64_t g0 = (int64_t)now.group * a.N * (GATED ? 2 : 1) + col;
      const bool biased = has_bias(a.epi);
      const float xs = Elem<T>::kInt ? a.xs[a.gather ? q / a.per : row] : 1.0f;
      auto z = [&](int jj, int64_t at) __attribute__((always_inline)) {
        Acc s = sums[parity][0][2 * i + jj][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += sums[parity][w][2 * i + jj][lane];
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
      f32x4 v = z(j, g0);
      with_activation(a.epi, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = activated<decltype(act)::value>(v[e]);
      });
      if constexpr (GATED) v *= z(1, g0 + a.N);
      TOut* out = (TOut*)a.C + to * a.ldc + col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col + e >= a.N) continue;
        if (!GATED && a.R) v[e] += to_f32(((const TOut*)a.R)[to * a.ldr + col + e]);
        out[e] = from_f32<TOut>(v[e]);
      }
    }
    parity ^= 1;
  };
  constexpr int OPS = BN / 8 + 2 * TM;
  static_for<P - 1>([&](auto j) __attribute__((always_inline)) { issue(j); });
  int todo = (int)(f1 - f0) * pieces, rest = pieces;
  while (todo > 0)
    static_for<P>([&](auto j) __attribute__((always_inline)) {
      if (todo > 0) {
        issue(std::integral_constant<int, (decltype(j)::value + P - 1) % P>{});
        // (what else was issued meanwhile only makes the wait longer)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((P - 1) * OPS));
        asm volatile("" ::: "memory");
        multiply(j);
        --todo;
        if (--rest == 0) {
          rest = pieces;
          write();
          now.next(a);
          if (now.tiles == 0) todo = 0;
        }
      }
    });
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));  // (the last pieces' zeros)
}

template <typename T, typename TOut, int BM, int BN, int P, bool PAST>
hipError_t launch_tiles(Args a, bool gated, hipStream_t stream) {
  const int cols = gated ? BN / 2 : BN;
  a.tiles_n = (a.N + cols - 1) / cols;
  // tiles of rows of all groups: what their ends can add
  const int64_t tiles_m = a.offsets ? a.rows / BM + std::min(a.groups, a.rows) : (a.rows + BM - 1) / BM;
  const dim3 grid((uint32_t)(tiles_m * a.tiles_n)), block(256);
  if (gated) hipLaunchKernelGGL((tile_kernel<T, TOut, true, BM, BN, P, PAST>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((tile_kernel<T, TOut, false, BM, BN, P, PAST>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// Workgroups that stay: two a CU.
template <typename T, typename TOut, bool PAST>
hipError_t launch_stream(Args a, bool gated, hipStream_t stream) {
  constexpr int BM = 16, P = 4;
  const int cols = gated ? 16 : 32;
  a.tiles_n = (a.N + cols - 1) / cols;
  const int64_t tiles_m = a.offsets ? a.rows / BM + std::min(a.groups, a.rows) : (a.rows + BM - 1) / BM;
  const dim3 grid((uint32_t)std::min<int64_t>(tiles_m * a.tiles_n, 512)), block(256);
  if (gated) hipLaunchKernelGGL((stream_kernel<T, TOut, true, BM, P, PAST>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((stream_kernel<T, TOut, false, BM, P, PAST>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// The kernel, by what the host knows: the rows a group has on average, the bytes
// of a row of K and those of all weights, and how many tiles there are for 256
// CUs.  Measured (us; W past the caches where it has 128 MiB):
//   stream: up to 4 rows a group (16 of a single one) and K of 4 KiB.  2 rows, 64
//     groups of 2 x 1024 x 2048 bf16 80.3, 64 x 64 88.0; K of 2 KiB 43.2 and 40.7.
//     i8, 16 x 2048 x 8192 10.1 and 12.4, 16 x 4096 x 4096 7.5 and 8.3.  (Its tiles
//     of 16 rows are the faster ones for more rows too while few columns leave
//     CUs idle: 64 x 2048 x 8192 10.3 and 13.5, 32 x 4096 x 4096 7.5 and 8.5, but 64 x
//     4096 x 4096 10.1 and 8.9, 64 x 8192 x 8192 39.3 and 14.8.)
//   256 x 256: more than 96 rows, K of 2 KiB, tiles for most CUs (more than 176 of
//     256; 192 tiles, i8 2880 x 4096 x 2048 31.2, 128 x 128 32.8; 176, 2816 rows 30.6
//     and 32.7, and 2048 x 5632 x 4096 48.0 and 56.4: the border could be lower).  i8
//     4096 x 4096 x 4096 53.8, 128 x 128 68.3; K of 1 KiB 33.6 and 32.4; 2048 x 4096 x
//     4096 44.0 and 35.9; 32 groups of 512 rows x 2048 x 1024 bf16 97.2 and 104; 64
//     rows a group 131 and 126.
//   128 x 128, two a CU: more than 48 rows, K of 1 KiB, more than one a CU.  i8 4096
//     x 4096 x 1024 32.4, 64 x 64 38.9; K of 256 24.7 and 24.5; 32 rows a group 122
//     and 94.5.  Of four stages where one a CU is enough for all, more than 160:
//     1024 x 4096 x 4096 21.1, of two stages 25.2, 64 x 64 26.5; 1024 x 2560 x 4096, 160
//     tiles, 17.6 and (64 x 64) 19.5, 512 x 4096 x 4096, 128 tiles, 17.3 and 15.2: the
//     border could be lower by some tiles.
//   64 x 64: the rest, four a CU of two stages where there are many (and K below 4
//     KiB, or more than 48 rows) or K is short, else two of four stages.  i8 1001 x
//     2055 x 4096 20.7 and 22.3, 800 x 4096 x 4096 25.7 and 25.6; 7252 x 470 x 176 7.7 and 11.0, 128 x 128 13.3; 256
//     x 4096 x 4096 16.9 and 9.5; 32 rows a group of K of 4 KiB 121 and 94.6.
// Weights of 128 MiB and more are read past the caches (64 x 64, 32 rows: 94.5 for
// 107.7), unless a group's many rows read them often (2048 rows, 862 for 876);
// fewer may still be in the last-level cache (i8, 16 x 8192 x 8192, called in
// turn: 13.3, past it 14.6).
template <typename T, typename TOut>
hipError_t launch(const Args& a, bool gated, hipStream_t stream) {
  const int64_t groups = std::min(a.groups, a.rows), average = (a.rows + groups - 1) / groups;
  const int64_t cols = (int64_t)a.N * (gated ? 2 : 1), row = (int64_t)a.K * sizeof(T);
  const bool past = groups * cols * row >= ((int64_t)128 << 20);
  auto tiles = [&](int bm, int bn) { return groups * ((average + bm - 1) / bm) * ((cols + bn - 1) / bn); };
  if (average <= (a.offsets ? 4 : 16) && row >= 4096)
    return past ? launch_stream<T, TOut, true>(a, gated, stream) : launch_stream<T, TOut, false>(a, gated, stream);
  if (average > 96 && row >= 2048 && tiles(256, 256) > 176)
    return past && average <= 512 ? launch_tiles<T, TOut, 256, 256, 2, true>(a, gated, stream)
                                  : launch_tiles<T, TOut, 256, 256, 2, false>(a, gated, stream);
  if (average > 48 && row >= 1024 && tiles(128, 128) > 256)
    return past ? launch_tiles<T, TOut, 128, 128, 2, true>(a, gated, stream)
                : launch_tiles<T, TOut, 128, 128, 2, false>(a, gated, stream);
  if (average > 48 && row >= 4096 && tiles(128, 128) > 160)
    return launch_tiles<T, TOut, 128, 128, 4, false>(a, gated, stream);
  if (row <= 512 || (tiles(64, 64) > 512 && (row < 4096 || average > 48)))
    return past ? launch_tiles<T, TOut, 64, 64, 2, true>(a, gated, stream)
                : launch_tiles<T, TOut, 64, 64, 2, false>(a, gated, stream);
  return past ? launch_tiles<T, TOut, 64, 64, 4, true>(a, gated, stream)
              : launch_tiles<T, TOut, 64, 64, 4, false>(a, gated, stream);
}

// one translation unit per (input, output) format pair
hipError_t launch_f16_f16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_bf16_bf16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_i8_f16(const Args& a, bool gated, hipStream_t stream);
hipError_t launch_i8_bf16(const Args& a, bool gated, hipStream_t stream);

}  // namespace grouped
}  // namespace ge
