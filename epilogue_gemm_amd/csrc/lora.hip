// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//     C[m] = R[m] + s[a] (X[m] A[a]^T) B[a]^T        a = ids[m]
//
// Two kernels.  `shrink` forms the inner products U = X A^T (rank values a
// row) as fp32 partial sums over ranges of K; `expand` adds the partials in
// their order, brings U to the input format in two parts and does the second
// product for a range of columns.  Small problems take `expand` alone, which
// then forms U itself.  Rows come in any order of adapters: a workgroup takes
// 16 consecutive rows -- an MFMA operand -- and runs once over each adapter
// that occurs among them, keeping of each product the rows that are the
// adapter's; where tiles are few, the adapters of a tile are spread over
// workgroups (grid z).
//
// Measured and not kept: both products of a large problem in one kernel (4096
// x 4096 -> 4096, rank 64: 48 us against 41, as all of A and B pass through
// each CU); tiles of 32 rows (39 against 41 us, but 80 against 56 where each
// row has another adapter) and, for the second product, of 64; a second copy
// of the second product's loop for whole rows of one adapter, the next columns'
// loads in flight (41.8 against 43.6 us); eight waves a tile in the first
// product (42.6 against 41.9 us, 17.2 against 15.4 for 512 rows); three or
// four workgroups of `expand` a CU instead of two, by fewer registers and
// swizzled instead of padded rows in LDS (42.8 and 65.9 against 43.7 us, few
// rows 10.2 against 8.6); consecutive tiles on one XCD (16384 rows 112 against
// 99 us, rank 16).
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
};

// (a 16-byte access off its alignment is one instruction all the same)
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The adapter of a row, -1 for none.
__device__ __forceinline__ int row_adapter(const Args& a, int row) {
  const int id = row < a.M ? a.ids[row] : -1;
  return id >= 0 && id < a.adapters ? id : -1;
}

// f(adapter, rows) for each adapter among 16 rows, lane l having that of row
// l % 16, in the order of their first rows, rows a bit mask; uniform over the
// wave.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F&& f) {
  uint32_t todo = (uint32_t)__builtin_amdgcn_ballot_w64(id >= 0) & 0xffffu;
  while (todo) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t rows = (uint32_t)__builtin_amdgcn_ballot_w64(id == ad) & 0xffffu;
    todo &= ~rows;
    f(ad, rows);
  }
}

// U^T += A X^T over one of W waves' part of [kbeg, kend): first operand 16
// of the adapter's rows, second the 16 rows of X, so that lane (m = l % 16, h
// = l / 16) receives U[m][16 t + 4 h + e].  A wave's part is contiguous and
// taken in stages of 64 columns.  Loads take whole cache lines, eight rows of
// 128 bytes an instruction (sixteen half lines, an operand's own shape, cost
// the L1 twice as long), and change lanes through the wave's own LDS: 16-byte
// chunk x of row r at x ^ (r / 2 % 8), which keeps an operand's 16 rows on
// different banks.  The next stage's loads are in flight while one is
// multiplied (two or three more of them made it slower, 9.3 to 9.5 us for 16
// rows, K = 4096 in one kernel).  The waves' parts and the first stages (`turn`) of
// the ranges of K, or of the blocks of columns, lie apart, for the memory
// channels' sake; not those of the tiles, as a row's sums would then depend on
// where it stands (4096 rows, rank 64: 43.2 us, with them 43.5; each row another
// of 16 adapters: 289 and 378).
template <typename T, int RT, int W>
__device__ __forceinline__ void inner(const Args& a, f32x4 (&acc)[RT], int row0, int ad, int kbeg, int kend, char* lds,
                                      int wave, int lane, int turn) {
  const int lr = lane >> 3, lc = lane & 7, c = lane & 15, h = lane >> 4;
  const T* x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) x[j] = (const T*)a.X + (int64_t)min(row0 + 8 * j + lr, a.M - 1) * a.ldx + 8 * lc;
  const T* ab = (const T*)a.A + (int64_t)ad * a.rank * a.K;
  const uint32_t aoff = (uint32_t)lr * a.K + 8 * lc;
  const int part = (kend - kbeg + 64 * W - 1) / (64 * W) * 64;
  const int k1 = kbeg + part * wave, k2 = min(kend, k1 + part);
  const int stages = k2 > k1 ? (k2 - k1 + 63) / 64 : 0;
  if (stages == 0) return;
  u32x4 g[1 + RT][2];
  bool in;  // this lane's columns of the stage exist (K is a multiple of 8)
  int at = turn % stages;
  auto load = [&]() __attribute__((always_inline)) {
    const int k0 = k1 + 64 * at;
    if (++at == stages) at = 0;
    in = k0 + 8 * lc < k2;
    const int k = in ? k0 : -8 * lc;  // (else the row's first: a valid address)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      g[0][j] = *(const u32x4*)(x[j] + k);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        // eight rows exist or not together, as the rank is a multiple of 8
        const int r = 16 * t + 8 * j < a.rank ? 16 * t + 8 * j : 0;
        g[1 + t][j] = *(const u32x4*)(ab + (int64_t)r * a.K + (int64_t)k + aoff);
      }
    }
  };
  char* const w = lds + lr * 128 + ((lc ^ (lr >> 1)) << 4);
  char* const w1 = lds + (8 + lr) * 128 + ((lc ^ (4 + (lr >> 1))) << 4);
  const char* const rd = lds + c * 128;
  load();
  for (int n = 0; n < stages; ++n) {
    if (__builtin_amdgcn_ballot_w64(!in)) {
#pragma unroll
      for (int t = 0; t < 1 + RT; ++t)
        if (!in) g[t][0] = g[t][1] = u32x4{};
    }
#pragma unroll
    for (int t = 0; t < 1 + RT; ++t) {
      *(u32x4*)(w + 2048 * t) = g[t][0];
      *(u32x4*)(w1 + 2048 * t) = g[t][1];
    }
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS accesses are done in order)
    load();                           // (past the last stage: the first again)
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int chunk = ((4 * s + h) ^ (c >> 1)) << 4;
      const u32x4 xf = *(const u32x4*)(rd + chunk);
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = mfma16<T>(*(const u32x4*)(rd + 2048 * (1 + t) + chunk), xf, acc[t]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Eight values of a row of U, whose other pieces are in the next PIECES - 1
// lanes, in two 16-bit parts: scaled by 2^-ex, which brings the row's largest
// finite value into [1/2, 1), in f16, whose small values have fewer bits, into
// [2^14, 2^15), the rounded value and its rounded remainder (U's error is the
// result's: 2^-16 of a value in bf16, 2^-22 in f16 down to 2^-18 of the largest
// and 2^-39 of that below).  Returns ex.
template <typename T, int PIECES>
__device__ __forceinline__ int split(const float (&u)[8], u32x4& hi, u32x4& lo) {
  float mx = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(u[e]) < __builtin_inff() ? fabsf(u[e]) : 0.0f);
#pragma unroll
  for (int d = 1; d < PIECES; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  // (a row of zeros is left as it is)
  const int ex = mx > 0.0f ? max(__builtin_amdgcn_frexp_expf(mx), -120) - (__is_same(T, f16) ? 15 : 0) : 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v0 = __builtin_amdgcn_ldexpf(u[2 * e], -ex), v1 = __builtin_amdgcn_ldexpf(u[2 * e + 1], -ex);
    const T t0 = from_f32<T>(v0), t1 = from_f32<T>(v1);
    hi[e] = (uint32_t)bits16(t0) | (uint32_t)bits16(t1) << 16;
    // (the remainder of an infinity is no number: it has none)
    lo[e] = pack2_out<T>(fabsf(v0) < __builtin_inff() ? v0 - to_f32(t0) : 0.0f,
                         fabsf(v1) < __builtin_inff() ? v1 - to_f32(t1) : 0.0f);
  }
  return ex;
}

// U's partial sums.  Workgroup (tile, range, z) takes the adapters number z, z
// + Z, ... of its 16 rows; its four waves add up in LDS.
template <typename T, int RT>
__global__ __launch_bounds__(256) void shrink(Args a) {
  constexpr int RP = 16 * RT, PER = (1 + RT) * 2048;
  static_assert(16 * (RP + 1) * 4 <= PER, "a wave's sums take the place of its operands");
  __shared__ __attribute__((aligned(16))) char lds[4 * PER];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * 16;
  const int kbeg = blockIdx.y * a.kper, kend = min(a.K, kbeg + a.kper);
  uint32_t number = 0;
  each_adapter(row_adapter(a, row0 + c), [&](int ad, uint32_t rows) {
    if (number++ % gridDim.z != blockIdx.z) return;
    f32x4 acc[RT] = {};
    inner<T, RT, 4>(a, acc, row0, ad, kbeg, kend, lds + wave * PER, wave, lane, blockIdx.y);
    __syncthreads();  // every wave has read its operands: their place holds the sums
    float* red = (float*)(lds + wave * PER);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[c * (RP + 1) + 16 * t + 4 * h + e] = acc[t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * RP; i += 256) {
      const int m = i / RP, r = i % RP;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) sum += ((const float*)(lds + w * PER))[m * (RP + 1) + r];
      if (rows >> m & 1) a.U[((int64_t)blockIdx.y * a.M + row0 + m) * RP + r] = sum;
    }
    __syncthreads();  // the sums have been read
  });
}

// The second product, C^T = B U^T: first operand 16 rows of B (columns of C),
// second the 16 rows of U, so that lane (m, h) receives four columns of row m
// per product.  A workgroup has 16 rows and 64 columns a wave at a time; it
// adds up its rows' partials of U, eight values a thread, and leaves U's two
// parts in LDS.  ONE: no kernel before it, it forms U itself, its eight waves
// each an eighth of K.  The 64 rows of B of a wave are contiguous and loaded so,
// then change lanes through the wave's LDS; C changes lanes there too, so
// that R and C move in whole lines, eight rows of 128 bytes an instruction.
// The loads of the first columns are all issued before the first wait.
// Workgroup (tile, columns, z) takes the adapters number z, z + Z, ... of its
// rows, the first also the rows without one.  PAST: R and C are more than the
// caches hold and move past them.  Bound by R and C, and for small problems
// by the chain of ids, U and the LDS's two turns.
template <typename T, int RT, bool PAST, bool ONE>
__global__ __launch_bounds__(ONE ? 512 : 256) void expand(Args a) {
  constexpr int W = ONE ? 8 : 4;  // waves
  constexpr int RP = 16 * RT, ST = (RP + 31) / 32, LD = RP + 8;
  constexpr int PIECES = RP / 8, BL = 2 * RT;  // of a row of U; of a lane in 64 rows of B
  constexpr int PER2 = 64 * LD * 2 > 16 * 68 * 4 ? 64 * LD * 2 : 16 * 68 * 4;
  constexpr int PER = ONE && (1 + RT) * 2048 > PER2 ? (1 + RT) * 2048 : PER2;
  __shared__ __attribute__((aligned(16))) char lds[W * PER];
  __shared__ __attribute__((aligned(16))) uint16_t su[2][16][LD];
  __shared__ int sex[16], list[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane >> 3, lc = lane & 7, c = lane & 15, h = lane >> 4;
  const int row0 = blockIdx.x * 16;
  const int id = row_adapter(a, row0 + c);
  uint32_t mine = 0;  // the rows this workgroup writes
  int count = 0, first = 0;
  {
    uint32_t number = 0, some = 0;
    each_adapter(id, [&](int ad, uint32_t rows) {
      some |= rows;
      if (number++ % gridDim.z == blockIdx.z) {
        mine |= rows;
        if (threadIdx.x == 0) list[count] = ad;
        if (count++ == 0) first = ad;
      }
    });
    if (mine == 0 && blockIdx.z != 0) return;
    if (blockIdx.z == 0) mine |= ~some & 0xffffu;
  }
  if (mine == 0) return;  // (every row is another workgroup's)
  char* const wl = lds + wave * PER;
  const int pieces = a.rank >> 3;  // of a row of B
  u32x4 b[BL], r[2];
  auto load_b = [&](int ad, int n) __attribute__((always_inline)) {
    const T* p = (const T*)a.B + ((int64_t)ad * a.N + n) * a.rank;
    const int most = min(64, a.N - n) * pieces - 1;
#pragma unroll
    for (int i = 0; i < BL; ++i) b[i] = *(const u32x4*)(p + 8 * min(lane + 64 * i, most));
  };
  // R's rows 8 j + lr (for a row that is not ours, one that is; the columns
  // behind the last whole eight are read one by one below)
  auto load_r = [&](int n) __attribute__((always_inline)) {
    if (!a.R || a.N < 8) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int m = mine >> (8 * j + lr) & 1 ? 8 * j + lr : __builtin_ctz(mine);
      const T* p = (const T*)a.R + (int64_t)min(row0 + m, a.M - 1) * a.ldr + min(n + 8 * lc, a.N - 8);
      r[j] = PAST ? __builtin_nontemporal_load((const u32x4_any*)p) : *(const u32x4_any*)p;
    }
  };
  const int step = gridDim.y * 64 * W;
  int n0 = (blockIdx.y * W + wave) * 64;
  load_b(first, min(n0, a.N - 1));  // (no adapter: the first one's, not used)
  load_r(n0);
  const float back = id >= 0 && a.scale ? a.scale[id] : 1.0f;
  if constexpr (ONE) {
    // (at most one adapter: there is a workgroup for each)
    f32x4 acc[RT] = {};
    if (count > 0) inner<T, RT, W>(a, acc, row0, first, 0, a.K, wl, wave, lane, blockIdx.y);
    float* red = (float*)wl;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[c * (RP + 1) + 16 * t + 4 * h + e] = acc[t][e];
    __syncthreads();
    if (threadIdx.x < 16 * PIECES) {
      const int m = threadIdx.x / PIECES, x = threadIdx.x % PIECES * 8;
      float u[8] = {};
      // (past the rank stand other rows of A: zero, as an infinity times B's
      // zeros there would be NaN)
      if (x < a.rank) {
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] += ((const float*)(lds + w * PER))[m * (RP + 1) + x + e];
      }
      u32x4 hi, lo;
      const int ex = split<T, PIECES>(u, hi, lo);
      *(u32x4*)&su[0][m][x] = hi;
      *(u32x4*)&su[1][m][x] = lo;
      if (x == 0) sex[m] = ex;
    }
  } else if (threadIdx.x < 16 * PIECES) {
    const int m = threadIdx.x / PIECES, x = threadIdx.x % PIECES * 8;
    float u[8] = {};
    if (x < a.rank && row0 + m < a.M && (mine >> m & 1)) {
      const float* up = a.U + (int64_t)(row0 + m) * RP + x;
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
    u32x4 hi, lo;
    const int ex = split<T, PIECES>(u, hi, lo);
    *(u32x4*)&su[0][m][x] = hi;
    *(u32x4*)&su[1][m][x] = lo;
    if (x == 0) sex[m] = ex;
  }
  __syncthreads();
  const int ex = sex[c];
  u32x4 uh[ST], ul[ST];
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const int x = 32 * s + 8 * h;
    uh[s] = x < RP ? *(const u32x4*)&su[0][c][x] : u32x4{};
    ul[s] = x < RP ? *(const u32x4*)&su[1][c][x] : u32x4{};
  }
  for (; n0 < a.N; n0 += step) {
    f32x4 out[4] = {};
    for (int k = 0; k < count; ++k) {
      const int ad = __builtin_amdgcn_readfirstlane(list[k]);
      if (k > 0) load_b(ad, n0);
#pragma unroll
      for (int i = 0; i < BL; ++i)
        if (i < pieces) {
          const int q = lane + 64 * i, m = q / pieces;
          *(u32x4*)(wl + (m * LD + (q - m * pieces) * 8) * 2) = b[i];
        }
      __builtin_amdgcn_wave_barrier();  // (a wave's LDS accesses are done in order)
      u32x4 bf[4][ST];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < ST; ++s) bf[j][s] = *(const u32x4*)(wl + ((16 * j + c) * LD + min(32 * s + 8 * h, RP)) * 2);
      if (a.rank < 32 * ST) {  // past the rank: whatever stands there counts as zero
#pragma unroll
        for (int s = 0; s < ST; ++s)
          if (32 * s + 8 * h >= a.rank) bf[0][s] = bf[1][s] = bf[2][s] = bf[3][s] = u32x4{};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 acc = {};
#pragma unroll
        for (int s = 0; s < ST; ++s) {
          acc = mfma16<T>(bf[j][s], uh[s], acc);
          acc = mfma16<T>(bf[j][s], ul[s], acc);
        }
        if (id == ad) out[j] = acc;
      }
      __builtin_amdgcn_wave_barrier();
    }
    // C = R + 2^ex back out; the 16 x 64 change lanes: rows 8 j + lr
    float* const f = (float*)wl;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = id < 0 ? 0.0f : __builtin_amdgcn_ldexpf(out[j][e], ex) * back;
      *(f32x4*)(f + c * 68 + 16 * j + 4 * h) = x;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4 v0 = *(const f32x4*)(f + (8 * j + lr) * 68 + 8 * lc), v1 = *(const f32x4*)(f + (8 * j + lr) * 68 + 8 * lc + 4);
      float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
      const int row = row0 + 8 * j + lr, n = n0 + 8 * lc;
      if (row >= a.M || !(mine >> (8 * j + lr) & 1)) continue;
      T* cp = (T*)a.C + (int64_t)row * a.ldc + n;
      if (n + 8 <= a.N) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = a.R ? r[j][e] : 0u;
          w[e] = pack2_out<T>(v[2 * e] + to_f32(__builtin_bit_cast(T, (uint16_t)(x & 0xffffu))),
                              v[2 * e + 1] + to_f32(__builtin_bit_cast(T, (uint16_t)(x >> 16))));
        }
        if constexpr (PAST) __builtin_nontemporal_store(w, (u32x4_any*)cp);
        else *(u32x4_any*)cp = w;
      } else {
        const T* rp = a.R ? (const T*)a.R + (int64_t)row * a.ldr + n : nullptr;
        for (int e = 0; e < 8; ++e)
          if (n + e < a.N) cp[e] = from_f32<T>(v[e] + (rp ? to_f32(rp[e]) : 0.0f));
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (n0 + step < a.N) {
      load_b(first, n0 + step);
      load_r(n0 + step);
    }
  }
}

// Ranges of K, by the sizes alone.  Up to 1024 rows eight of 512 or more,
// which give the chip work (K = N = 4096, two kernels: 16 rows 8.7 us, one
// range 11.1; 512 rows, rank 64, 15.3 against 20.2).  More rows one, for the
// batches in which each row has another adapter, whose A then passes through a
// CU once a range and tile (2048 rows, rank 64: 139 us, two ranges 195; 4096
// rows 289 and 335).  Long runs of an adapter would rather have two up to 2048
// rows (1100 rows, rank 64: 23.9 and 20.7; 2000 rows 27.7 and 26.8) and gain
// nothing above (4096 rows, rank 64: 43.2, two 44.7, four 42.7; rank 16 29.2,
// 29.3, 30.6).
struct Cut {
  int tiles, ksplit, kper;
};
inline Cut cut(int64_t M, int64_t K) {
  const int64_t ks = M > 1024 ? 1 : K >= 4096 ? 8 : (K + 511) / 512;
  Cut s;
  s.tiles = (int)((M + 15) / 16);
  s.kper = (int)(((K + ks - 1) / ks + 255) / 256 * 256);
  s.ksplit = (int)((K + s.kper - 1) / s.kper);
  return s;
}

inline int64_t rank_pad(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Both products in one kernel: each workgroup then reads its adapter's whole
// A and its rows' whole X (`bytes`) by itself, against a second launch and
// U's way through memory.  That pays up to 320 KiB a workgroup and rank 64 (16
// rows, N = 4096: K = 1024, rank 16 6.7 us, two kernels 8.8; K = 2048, rank 64
// 9.1 and 9.9; K = 4096, rank 16 9.2 and 8.6 on the GPU, but 3 us less of the
// host; K = 4096, rank 64 12.7 and 9.5; K = 1024, rank 128 14.3 and 12.3),
// while all workgroups run at once and read no more than 80 MiB together (128
// rows, 512 workgroups, rank 16: K = 1024 8.9 and 11.5, K = 4096 13.3 and
// 11.8).
inline bool one(int64_t tiles, int64_t columns, int64_t adapters, int64_t bytes) {
  const int64_t wgs = tiles * columns * adapters;
  return bytes <= 320 << 10 && wgs <= 512 && wgs * bytes <= 80 << 20;
}

// Workgroups among which a tile's adapters are spread (grid z): as many as it
// can hold where tiles are few.  Those that find no adapter of theirs end at
// once; `expand`, whose rows cost more than its adapters, spreads less.
template <typename T, int RT>
hipError_t launch(const Args& a, const Cut& s, hipStream_t stream) {
  const int most = min(a.adapters, min(a.M, 16));
  if constexpr (RT <= 4) {
    const int y = (a.N + 511) / 512;
    if (one(s.tiles, y, most, (int64_t)(16 + 16 * RT) * a.K * 2)) {
      hipLaunchKernelGGL((expand<T, RT, false, true>), dim3(s.tiles, y, most), dim3(512), 0, stream, a);
      return hipGetLastError();
    }
  }
  const int z1 = s.tiles <= 4 ? most : s.tiles <= 256 ? min(most, 4) : 1;
  const int z2 = s.tiles <= 4 ? most : s.tiles <= 32 ? min(most, 4) : 1;
  hipLaunchKernelGGL((shrink<T, RT>), dim3(s.tiles, s.ksplit, z1), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns of a workgroup: 256, or more where that still leaves some 1024
  // workgroups; R and C beyond the L2s' 32 MiB go past the caches (4096 x 4096,
  // rank 64: 43.7 us against 48.8, with a reading of C after it 49.8 against
  // 54.8; 512 rows 16.7 against 15.7)
  const int y = min((a.N + 255) / 256, max(1, 1024 / s.tiles / z2));
  if ((int64_t)a.M * a.N * 4 > ((int64_t)32 << 20))
    hipLaunchKernelGGL((expand<T, RT, true, false>), dim3(s.tiles, y, z2), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((expand<T, RT, false, false>), dim3(s.tiles, y, z2), dim3(256), 0, stream, a);
  return hipGetLastError();
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
  // (a tile of 16 rows a workgroup of 256: a grid holds below 2^32 threads)
  if (rank > 128 || rank % 8 != 0 || K % 8 != 0 || M > kLim / 8 - 16 || K >= kLim / 8 || adapters > 65535 ||
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
  const ge::lora::Args a{X,   A,   B,   R,      scale,  ids,       C,           (float*)workspace,
                         ldx, ldr, ldc, (int)M, (int)N, (int)K,    (int)rank,   (int)adapters,
                         cut.ksplit, cut.kper};
  const hipError_t e = dtype == GEMM_EPI_F16 ? ge::lora::launch_rank<ge::f16>(a, cut, (hipStream_t)stream)
                                             : ge::lora::launch_rank<ge::bf16>(a, cut, (hipStream_t)stream);
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}

}  // extern "C"
