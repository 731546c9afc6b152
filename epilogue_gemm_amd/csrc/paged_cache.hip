// paged_cache.hip -- the paged key-value cache of a layer: the append of new
// tokens and the attention of one new token of each sequence over its pages,
//
//     O[i, h] = sum_j softmax_j(q . k_j / sqrt(D)) v_j     j < lens[i], page of j present
//
// with the keys of all sequences and heads split evenly over the workgroups
// that the chip holds at once (paged.hpp), and the pieces of a sequence that
// the split cuts joined by the workgroup that finishes last, or, where they
// are many, by a second kernel.  Bound by the cache's bytes (32 x 8192 bf16
// of mixed lengths, 8 heads of 128: 88 us, 6.0 TB/s), for few keys by the
// chain of lookups, loads and the join (1 x 1000: 8.3 us, 3 of them the join).
//
// For each piece -- some keys of one sequence, one key head and up to 16 of
// the query heads that share it -- the four waves of a workgroup take every
// fourth tile of 32 keys.  Both products are v_mfma_f32_16x16x32 chains whose
// operands come straight from memory and whose layouts meet without any
// movement between lanes (c = lane % 16, h = lane / 16):
//   * S^T = K Q^T: first operand 16 keys (lane c: key c, 8 values of it),
//     second the 16 query heads; lane (c, h) receives, for query head c,
//     the scores of keys 4 h + 0..3 of each group of 16;
//   * the probabilities of two groups are then the lane's second operand of
//     O^T = V^T P^T for 32 keys if the 32 places of the k axis are numbered
//     (h, u) -> key 16 (u / 4) + 4 h + u % 4;
//   * V^T's first operand for D / 16 products: lane (c, h) loads those eight
//     keys' values d = VEC c .. VEC c + VEC - 1 (VEC = D / 16; 16 lanes read
//     a whole row) and packs pairs of keys by v_perm; product j takes d =
//     VEC c + j.  Lane (c, h) ends with VEC consecutive values of query head
//     c's output for each e: d = VEC (4 h + e) + j.
#include "gemm_tile16.hpp"
#include "paged.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_decode.h"

namespace ge {
namespace paged {

using tile16::mfma16;

constexpr float kNegInf = -__builtin_inff();

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendArgs {
  char *k, *v;  // the cache
  float *ks, *vs;
  const int32_t *pages, *lens, *starts;
  const void *K, *V;
  int64_t ld, ldk, ldv;
  int num_pages, page_size, heads, width, batch, tokens;
};

// The smallest integer e >= -100 with amax <= 448 * 2^e, for a finite amax:
// amax = m 2^k, m in [1/2, 1), and 448 = 0.875 * 2^9.
__device__ __forceinline__ int scale_exponent(float amax) {
  const int k = __builtin_amdgcn_frexp_expf(amax);
  const int e = k - (__builtin_amdgcn_frexp_mantf(amax) > 0.875f ? 8 : 9);
  return amax == 0.0f ? -100 : max(e, -100);
}

// One wave a token: the first rows' loads, then the token's sequence, page
// and slot while they are in flight, then the rows of all heads, 8 values a
// lane.  An E4M3 row's largest value is found over the D / 8 lanes that hold
// it, by the bits of |x|, which order a NaN above every number.  Bound by
// memory for many tokens, by the three dependent lookups for few.
template <typename T, bool FP8, int D, bool PAST>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  constexpr int LPR = D / 8;   // lanes of a row
  constexpr int BATCH = 4;     // pieces of a lane in flight
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t >= a.tokens) return;
  const int n = a.heads * LPR;  // pieces of K, then as many of V
  const T* k = (const T*)a.K + t * a.ldk;
  const T* v = (const T*)a.V + t * a.ldv;
  u32x4 x[BATCH];
  auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int i = min(i0 + 64 * b, 2 * n - 1);  // (past the last: it again)
      const u32x4* p = (const u32x4*)(i >= n ? v + 8 * (i - n) : k + 8 * i);
      x[b] = PAST ? __builtin_nontemporal_load(p) : *p;
    }
  };
  load(lane);
  int seq = t, end = t + 1;
  if (a.starts) {
    // the number of sequences whose rows end at or before this one
    seq = 0;
    for (int i = 0; i < a.batch; i += 64) {
      const bool past = i + lane < a.batch && a.starts[i + lane + 1] <= t;
      seq += __builtin_popcountll(__builtin_amdgcn_ballot_w64(past));
    }
    if (seq >= a.batch || a.starts[0] > t) return;
    end = a.starts[seq + 1];
  }
  const int pos = new_position(a.lens[seq], end, t, a.width * a.page_size);
  if (pos < 0) return;
  const int page = page_or_none(a.pages[seq * a.ld + pos / a.page_size], a.num_pages);
  if (page < 0) return;
  const int64_t row0 = row_of(page, a.heads, 0, a.page_size, pos % a.page_size);
  for (int i0 = lane; i0 < 2 * n; i0 += 64 * BATCH) {
    if (i0 != lane) load(i0);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int i = i0 + 64 * b;
      if (i >= 2 * n) break;
      const bool val = i >= n;
      const int j = val ? i - n : i, head = j / LPR, at = j % LPR;
      const int64_t row = row0 + (int64_t)head * a.page_size;
      char* dst = val ? a.v : a.k;
      if constexpr (!FP8) {
        *(u32x4*)(dst + (row * D + 8 * at) * 2) = x[b];
      } else {
        float f[8];
        uint32_t mx = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          f[2 * w] = to_f32(__builtin_bit_cast(T, (uint16_t)(x[b][w] & 0xffffu)));
          f[2 * w + 1] = to_f32(__builtin_bit_cast(T, (uint16_t)(x[b][w] >> 16)));
          mx = max(mx, max(__builtin_bit_cast(uint32_t, f[2 * w]) & 0x7fffffffu,
                           __builtin_bit_cast(uint32_t, f[2 * w + 1]) & 0x7fffffffu));
        }
        // (whole groups of lanes have a row or none)
        const float amax = __builtin_bit_cast(float, wave::max_over<LPR>(mx));
        const int e = scale_exponent(amax);
        const bool number = amax < __builtin_inff();
        const float inv = number ? __builtin_amdgcn_ldexpf(1.0f, -e) : __builtin_nanf("");
        // (within +-448, by the scale: no clamp)
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
        *(u32x2*)(dst + row * D + 8 * at) = u32x2{(uint32_t)lo, (uint32_t)hi};
        if (at == 0) (val ? a.vs : a.ks)[row] = number ? __builtin_amdgcn_ldexpf(1.0f, e) : __builtin_nanf("");
      }
    }
  }
}

// ---------------------------------------------------------------------------
// decode attention
// ---------------------------------------------------------------------------
// Workgroups of the decode attention: those the memory system wants in flight
// at once.  Rows of 128 bytes and more: one for each of the 256 CUs (its waves
// then have 32 to 128 KiB in flight; 1 x 131072 bf16, D = 128: 89 us, two for
// each 95; 8 x 65536 E4M3, D = 128: 100 and 102; 32 x 8192 and 128 x 2047 f16, D
// = 64, the same); shorter rows: up to two (16 x 32768 E4M3, D = 64: 53 against
// 60 us).  A third tile in flight was no faster.
constexpr int kWorkgroups = 512;
inline int workgroups_for(int row_bytes) { return row_bytes >= 128 ? 256 : kWorkgroups; }
static_assert(kWorkgroups * 4 == GEMM_EPI_ATTENTION_DECODE_COUNTER_BYTES, "a counter each");
static_assert(kWorkgroups <= 512, "share_begin");

struct DecodeArgs {
  const char *k, *v;
  const float *ks, *vs;
  const int32_t *pages, *lens;
  const void* Q;
  void* O;
  unsigned* arrivals;  // kWorkgroups counters, zero between runs
  float* part;  // two pieces per workgroup: 16 x D sums, then 16 x (maximum, sum)
  int64_t ld, ldq, ldo;
  int num_pages, page_size, heads, width, batch;
  int group;   // query heads per key head
  int qtiles;  // tiles of 16 of them
  int workgroups;
  Divider groups;  // by the groups of 16 tokens of a page
  float scale_log2;
};

// The batch's units, counted by each wave for itself: lane l for sequences
// l * per .. + per - 1.
struct Units {
  int per, i0, i1;  // this lane's sequences
  int len;          // tokens of the first of them
  int own, before;  // units of this lane's sequences, and of those before them
  int total;
  bool empty;  // some sequence of the batch has no tokens
};
__device__ __forceinline__ Units count_units(const int32_t* lens, int batch, int cap, int lane) {
  Units s;
  s.per = (batch + 63) / 64;
  s.i0 = min(lane * s.per, batch);
  s.i1 = min(s.i0 + s.per, batch);
  s.own = s.len = 0;
  bool none = false;
  for (int i = s.i0; i < s.i1; ++i) {
    const int n = seq_len(lens[i], cap);
    if (i == s.i0) s.len = n;
    none |= n == 0;
    s.own += units_of(n);
  }
  const int incl = wave::scan(s.own);
  s.before = incl - s.own;
  s.total = __builtin_amdgcn_readlane(incl, 63);
  s.empty = __builtin_amdgcn_ballot_w64(none) != 0;
  return s;
}
// Tokens of sequence seq (the same in every lane): from the lanes where each
// has one.
__device__ __forceinline__ int len_of(const Units& un, const int32_t* lens, int seq, int cap) {
  return un.per == 1 ? __builtin_amdgcn_readlane(un.len, seq)
                     : __builtin_amdgcn_readfirstlane(seq_len(lens[seq], cap));
}

// Piece `which` of share w: 0 of a sequence that began in an earlier
// workgroup's share, 1 of one that begins in this one's and ends later.
template <int D>
__device__ __forceinline__ float* part_of(const DecodeArgs& a, int w, int which) {
  return a.part + ((int64_t)w * 2 + which) * (16 * (D + 2));
}

// Joins `rows` rows from `row0` on of a cut sequence's pieces, in their
// order, into o[row - row0][D]: a row is D / 4 threads', and what threads
// remain make further groups that take every n-th piece each and add up in
// LDS (256 x 6 floats), so that many loads are in flight.  rows * D / 4 <= 256.
template <typename T, int D>
__device__ __forceinline__ void join_rows(const DecodeArgs& a, int w0, int pieces, int row0, int rows, T* o, float* lds) {
  constexpr int LPR = D / 4;
  const int slots = rows * LPR, groups = 256 / slots;
  const int g = threadIdx.x / slots, slot = threadIdx.x % slots, row = row0 + slot / LPR, t = slot % LPR;
  float m = kNegInf, l = 0.0f;
  f32x4 s = {};
  auto add = [&](float mp, float lp, f32x4 sp) __attribute__((always_inline)) {
    const float mn = fmaxf(m, mp), ref = mn == kNegInf ? 0.0f : mn;
    const float x = __builtin_amdgcn_exp2f(m - ref), y = __builtin_amdgcn_exp2f(mp - ref);
    m = mn;
    l = l * x + lp * y;
    s = s * x + sp * y;
  };
  if (g < groups) {
    // a round's loads at a time (past the last piece: a maximum of -inf)
    for (int p0 = g; p0 < pieces; p0 += kBatch * groups) {
      float mp[kBatch], lp[kBatch];
      f32x4 sp[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = min(p0 + i * groups, pieces - 1);
        const float* pp = part_of<D>(a, w0 + p, p == 0);
        mp[i] = p0 + i * groups < pieces ? pp[16 * D + 2 * row] : kNegInf;
        lp[i] = pp[16 * D + 2 * row + 1];
        sp[i] = *(const f32x4*)(pp + row * D + 4 * t);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add(mp[i], lp[i], sp[i]);
    }
    f32x4* ls = (f32x4*)lds + threadIdx.x;
    *ls = s;
    lds[1024 + 2 * threadIdx.x] = m;
    lds[1024 + 2 * threadIdx.x + 1] = l;
  }
  __syncthreads();
  if (g == 0) {
    for (int i = 1; i < groups; ++i) {
      const int th = i * slots + slot;
      add(lds[1024 + 2 * th], lds[1024 + 2 * th + 1], ((const f32x4*)lds)[th]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *(u32x2*)(o + (row - row0) * D + 4 * t) = u32x2{pack2_out<T>(s[0] * inv, s[1] * inv), pack2_out<T>(s[2] * inv, s[3] * inv)};
  }
}

// All rows of a cut sequence's pieces.
template <typename T, int D>
__device__ __forceinline__ void join_pieces(const DecodeArgs& a, int w0, int pieces, int rows, T* o, float* lds) {
  constexpr int most = 1024 / D;  // rows at a time
  for (int r = 0; r < rows; r += most) {
    join_rows<T, D>(a, w0, pieces, r, min(most, rows - r), o + r * D, lds);
    __syncthreads();  // the sums in LDS have been read
  }
}

// 8-bit codes 2 HI and 2 HI + 1 of src as two 16-bit values, times the
// power of two `scale`
template <typename T, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t src, float scale) {
  if constexpr (__is_same(T, f16))
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(src, scale, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(src, scale, HI));
}

// A tile of 32 keys as loaded: of each group of 16, whose K rows are
// contiguous, this lane's 16 bytes of every KiB; (u = 4 g + 0..3) this lane's
// part of V's rows; and how many of the group's keys exist.
template <bool FP8, int D>
struct Tile {
  static constexpr int VEC = D / 16;        // values of a row per lane in V's operand
  static constexpr int EB = FP8 ? 1 : 2;    // bytes of a cache element
  static constexpr int RB = D * EB;         // bytes of a cache row
  static constexpr int KL = RB / 64;        // KiB of a group's K
  static constexpr int VW = VEC * EB / 4;   // 32-bit words of a lane for one key's V
  typedef uint32_t vwords __attribute__((ext_vector_type(VW == 1 ? 2 : VW)));  // (one word: in .x)
  u32x4 k[2][KL];
  vwords v[8];
  f32x4 ks[2], vs[2];
  int valid[2];
};

template <typename T, bool FP8, int D>
__global__ __launch_bounds__(256, 2) void decode_kernel(DecodeArgs a) {
  using Tl = Tile<FP8, D>;
  constexpr int VEC = Tl::VEC, EB = Tl::EB, KL = Tl::KL, VW = Tl::VW, RB = Tl::RB;
  constexpr int KS = D / 32;  // 32-deep steps of a score
  // f16 does not hold every code times its scale (65504 is held as 256 times
  // 2^8, and small rows lie below 2^-14).  Beside f16 queries K's codes enter
  // their product as they are and the scores take the scales; the second product
  // of an 8-bit cache is bf16's, which has room for all of V's.
  constexpr bool kCodes = FP8 && __is_same(T, f16);
  typedef std::conditional_t<FP8, bf16, T> TV;
  // The weights are taken relative to 2^-7 of the largest in f16, which has
  // fewer bits below 2^-14: there are the weights of most keys beside one that
  // stands out (one of 2^-17 was off by up to 0.5 %).  The two parts then lose
  // 2^-22 of a weight of 2^-10 of the largest and more, and 2^-32 of the largest
  // of smaller ones; no weight is above 2^8, however maximum - 7 is rounded.
  constexpr float kAbove = __is_same(TV, f16) ? 7.0f : 0.0f;
  __shared__ float sm[4][16], sl[4][16];
  __shared__ __attribute__((aligned(16))) float so[4][16][D + 4];
  __shared__ int last_arrived;
  // K's rows change lanes through LDS, each wave's in its own part: loaded in
  // whole KiB, read as MFMA operands (lane (c, h): 16 bytes of row c).  Chunk
  // x of row r stands at x ^ (r RB / 256), so that the 16 rows of a read fall
  // on different banks.
  __shared__ __attribute__((aligned(1024))) char sk[4][32 * RB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int cap = a.width * a.page_size;

  const int columns = a.heads * a.qtiles;
  const Units un = count_units(a.lens, a.batch, cap, lane);
  // an empty sequence has no units: its zeros are written here
  if (un.empty)
    for (int i = blockIdx.x; i < a.batch * columns; i += gridDim.x) {
      const int seq = i / columns, col = i % columns;
      if (seq_len(a.lens[seq], cap) != 0) continue;
      const int qh = (col % a.qtiles) * 16 + (threadIdx.x >> 4), d0 = (threadIdx.x & 15) * VEC;
      if (qh >= a.group) continue;
      T* op = (T*)a.O + seq * a.ldo + (int64_t)((col / a.qtiles) * a.group + qh) * D + d0;
#pragma unroll
      for (int j = 0; j < VEC; j += 2) *(uint32_t*)(op + j) = 0u;
    }
  const Shares sh = make_shares(un.total * columns, workgroups_of(un.total * columns, gridDim.x));
  if ((int)blockIdx.x >= sh.n) return;
  const int w = share_at(sh, blockIdx.x);
  int f = share_begin(sh, w);
  const int fend = share_begin(sh, w + 1);
  int column = (int)((uint32_t)f / (uint32_t)un.total), u = f - column * un.total;  // unit u of this column is next
  // its sequence: the lane that counted it walks there
  int seq, begin;  // the sequence, and the number of its first unit in a column
  {
    const uint64_t owner = __builtin_amdgcn_ballot_w64(u >= un.before && u < un.before + un.own);
    int i = un.i0, at = un.before;
    while (i < un.i1) {
      const int n = units_of(seq_len(a.lens[i], cap));
      if (u < at + n) break;
      at += n;
      ++i;
    }
    const int src = __builtin_ctzll(owner);
    seq = __builtin_amdgcn_readlane(i, src);
    begin = __builtin_amdgcn_readlane(at, src);
  }
  while (f < fend) {
  const int len = len_of(un, a.lens, seq, cap), units = units_of(len);
  if (units == 0) {
    if (++seq == a.batch) {
      seq = 0;
      ++column;
      begin = u = 0;
    }
    continue;
  }
  const int take = min(fend - f, begin + units - u);
  const int kbeg = (u - begin) * kUnit, kend = min(len, kbeg + take * kUnit);

  // the query heads of this column
  const int head = column / a.qtiles, first = (column % a.qtiles) * 16;
  const bool query = first + c < a.group;
  const T* q = (const T*)a.Q + seq * a.ldq + (int64_t)(head * a.group + first + c) * D;
  u32x4 qf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    // the 8 values of a row that lane (., h) multiplies in step s
    const int d = FP8 ? 64 * (s >> 1) + 16 * h + 8 * (s & 1) : 32 * s + 8 * h;
    qf[s] = query ? *(const u32x4*)(q + d) : u32x4{};
  }

  f32x4 acc[VEC] = {};
  float m = kNegInf, l = 0.0f;
  const int32_t* table = a.pages + seq * a.ld;
  // this wave's tiles are 128 keys apart
  const int k1 = kbeg + 32 * wave, last = k1 < kend ? (kend - 1 - k1) / 128 : -1;
  // The pages of 32 tiles at a time: lane 2 i + g has that of group g of the
  // i-th (past the end: of the tile's first, whose keys are then masked).
  // Looked up here, no tile's loads wait behind a lookup.
  int entries = -1;
  auto look_up = [&](int n) __attribute__((always_inline)) {
    const int k = looked_up_key(k1, kend, last, n + (lane >> 1), lane & 1);
    entries = k >= 0 ? page_or_none(table[divide(k >> 4, a.groups)], a.num_pages) : -1;
  };
  constexpr int CPR = RB / 16;  // chunks of a row
  auto kwrite = [&](int i) __attribute__((always_inline)) {
    const int r = lane / CPR + i * (1024 / RB);
    return r * RB + (((lane % CPR) ^ (r * RB / 256 % CPR)) << 4);
  };
  auto kread = [&](int i) __attribute__((always_inline)) { return c * RB + (((4 * i + h) ^ (c * RB / 256 % CPR)) << 4); };
  const uint32_t koff = (uint32_t)(16 * lane), voff = (uint32_t)(4 * h * D * EB + c * VEC * EB);
  // Tile n of this wave; past the last one its first lines, which the loop
  // below does not use (loads that are not always issued would make every wait
  // a wait for all of them).
  auto load = [&](Tl& t, int n) __attribute__((always_inline)) {
    if (n <= last && n % 32 == 0) look_up(n);
    const int i = min(n, last), k0 = k1 + 128 * i;
    const uint32_t ko = n > last ? 0 : koff, vo = n > last ? 0 : voff;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int gk = k0 + 16 * g, at = gk < kend ? gk : k0;
      const int page = __builtin_amdgcn_readlane(entries, 2 * (i & 31) + g);
      t.valid[g] = page < 0 ? 0 : max(0, min(kend - gk, 16));
      const int64_t row =
          row_of(max(page, 0), a.heads, head, a.page_size, at - divide(at >> 4, a.groups) * a.page_size);
      const char* kp = a.k + row * (D * EB);
      const char* vp = a.v + row * (D * EB);
#pragma unroll
      for (int i = 0; i < KL; ++i) t.k[g][i] = __builtin_nontemporal_load((const u32x4*)(kp + ko + 1024 * i));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const char* r = vp + vo + u * D * EB;
        if constexpr (VW == 1) t.v[4 * g + u].x = *(const uint32_t*)r;
        else t.v[4 * g + u] = __builtin_nontemporal_load((const typename Tl::vwords*)r);
      }
      if constexpr (FP8) {
        if constexpr (kCodes) t.ks[g] = *(const f32x4*)(a.ks + row + 4 * h);
        else t.ks[g].x = a.ks[row + c];
        t.vs[g] = *(const f32x4*)(a.vs + row + 4 * h);
      }
    }
  };
  auto multiply = [&](const Tl& t) __attribute__((always_inline)) {
    const bool whole = t.valid[0] == 16 && t.valid[1] == 16;
    // scores
    char* const kl = sk[wave];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < KL; ++i) *(u32x4*)(kl + g * 16 * RB + kwrite(i)) = t.k[g][i];
    __builtin_amdgcn_wave_barrier();  // (a wave's LDS accesses are done in order)
    f32x4 s[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      s[g] = f32x4{};
      u32x4 kf[KL];
#pragma unroll
      for (int i = 0; i < KL; ++i) kf[i] = *(const u32x4*)(kl + g * 16 * RB + kread(i));
      if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
          const u32x4 x = kf[i];
          const float f = kCodes ? 1.0f : t.ks[g].x;
          const u32x4 lo = {widen2<T, false>(x[0], f), widen2<T, true>(x[0], f), widen2<T, false>(x[1], f),
                            widen2<T, true>(x[1], f)};
          const u32x4 hi = {widen2<T, false>(x[2], f), widen2<T, true>(x[2], f), widen2<T, false>(x[3], f),
                            widen2<T, true>(x[3], f)};
          s[g] = mfma16<T>(lo, qf[2 * i], s[g]);
          s[g] = mfma16<T>(hi, qf[2 * i + 1], s[g]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < KL; ++i) s[g] = mfma16<T>(kf[i], qf[i], s[g]);
      }
      if constexpr (kCodes) s[g] *= t.ks[g] * a.scale_log2;
      else s[g] *= a.scale_log2;
    }
    if (!whole) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * h + e >= t.valid[g]) s[g][e] = kNegInf;
    }
    // the reference of the weights: the running maximum of the query head over
    // all four quarters, less kAbove; the sums are rescaled only when some
    // head's moves
    float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                     fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    mx = wave::over_rows<wave::Max>(mx);
    if constexpr (kAbove != 0.0f) mx -= kAbove;
    if (__builtin_amdgcn_ballot_w64(mx > m)) {
      const float mn = fmaxf(m, mx);
      const float alpha = __builtin_amdgcn_exp2f(m - (mn == kNegInf ? 0.0f : mn));
      m = mn;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= alpha;
    }
    const float ref = m == kNegInf ? 0.0f : m;
    // probabilities, in two parts (fp32 products have a sixteenth of the rate;
    // one 16-bit part alone would be off by as much as the output's rounding:
    // two lose 2^-16 of each weight in bf16, a 256th of that rounding)
    u32x4 ph, pl;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float p0 = __builtin_amdgcn_exp2f(s[w >> 1][2 * (w & 1)] - ref);
      const float p1 = __builtin_amdgcn_exp2f(s[w >> 1][2 * (w & 1) + 1] - ref);
      l += p0 + p1;
      const TV t0 = from_f32<TV>(p0), t1 = from_f32<TV>(p1);
      ph[w] = (uint32_t)bits16(t0) | (uint32_t)bits16(t1) << 16;
      pl[w] = pack2_out<TV>(p0 - to_f32(t0), p1 - to_f32(t1));
    }
    // V: this lane's eight keys, 16-bit
    uint32_t vr[8][VEC / 2];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if constexpr (FP8) {
        const float f = t.vs[u >> 2][u & 3];
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          vr[u][2 * w] = widen2<TV, false>(t.v[u][w], f);
          vr[u][2 * w + 1] = widen2<TV, true>(t.v[u][w], f);
        }
      } else {
#pragma unroll
        for (int w = 0; w < VW; ++w) vr[u][w] = t.v[u][w];
      }
    }
    // a key without a page or past the end: its V may hold anything, and zero
    // times anything need not be zero
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (4 * h + (u & 3) >= t.valid[u >> 2]) {
#pragma unroll
          for (int w = 0; w < VEC / 2; ++w) vr[u][w] = 0u;
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      u32x4 vf;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        vf[w] = __builtin_amdgcn_perm(vr[2 * w + 1][j >> 1], vr[2 * w][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
      acc[j] = mfma16<TV>(vf, ph, acc[j]);
      acc[j] = mfma16<TV>(vf, pl, acc[j]);
    }
  };
  // The next tile's loads are in flight while one is multiplied.
  if (last >= 0) {
    Tl t0, t1;
    load(t0, 0);
    for (int n = 0;; n += 2) {
      load(t1, n + 1);
      multiply(t0);
      if (n + 1 > last) break;
      load(t0, n + 2);
      multiply(t1);
      if (n + 2 > last) break;
    }
  }

  // join the four waves
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (h == 0) {
    sm[wave][c] = m;
    sl[wave][c] = l;
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) so[wave][c][VEC * (4 * h + e) + j] = acc[j][e];
  __syncthreads();
  const int rows = min(16, a.group - first);
  for (int p = threadIdx.x; p < rows * (D / 2); p += 256) {  // two values each
    const int qh = p / (D / 2), d = p % (D / 2) * 2;
    const float mj = fmaxf(fmaxf(sm[0][qh], sm[1][qh]), fmaxf(sm[2][qh], sm[3][qh]));
    const float ref = mj == kNegInf ? 0.0f : mj;
    float o0 = 0.0f, o1 = 0.0f, lj = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __builtin_amdgcn_exp2f(sm[i][qh] - ref);
      lj += x * sl[i][qh];
      o0 += x * so[i][qh][d];
      o1 += x * so[i][qh][d + 1];
    }
    if (take == units) {
      const float inv = lj == 0.0f ? 0.0f : 1.0f / lj;
      *(uint32_t*)((T*)a.O + seq * a.ldo + (int64_t)(head * a.group + first + qh) * D + d) = pack2_out<T>(o0 * inv, o1 * inv);
    } else {
      // (agent-scope stores reach the level that all XCDs share)
      auto store = [](float* to, float x, float y) __attribute__((always_inline)) {
        __hip_atomic_store((uint64_t*)to, (uint64_t)__builtin_bit_cast(uint32_t, x) | (uint64_t)__builtin_bit_cast(uint32_t, y) << 32,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      float* pp = part_of<D>(a, w, u == begin);
      store(pp + qh * D + d, o0, o1);
      if (d == 0) store(pp + 16 * D + 2 * qh, mj, lj);
    }
  }
  const int f0 = f - (u - begin);
  const int w0 = share_of(sh, f0), pieces = take == units ? 1 : share_of(sh, f0 + units - 1) - w0 + 1;
  if (take != units && joined_here(pieces, rows, D)) {
    // Count the piece at the sequence's counter (that of the workgroup in
    // whose share it begins: a share holds the beginning of at most one cut
    // sequence); the last to arrive joins the pieces, in their order, and
    // clears the counter for the next run.  As in the split products: every
    // thread's stores are acknowledged before the count (a fence that
    // releases would write back the XCD's whole L2), and the joining
    // workgroup acquires at agent scope after it.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    if (threadIdx.x == 0)
      last_arrived = __hip_atomic_fetch_add(a.arrivals + w0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                     (unsigned)(pieces - 1);
    __syncthreads();
    if (last_arrived) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      if (threadIdx.x == 0) __hip_atomic_store(a.arrivals + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      join_pieces<T, D>(a, w0, pieces, rows,
                        (T*)a.O + seq * a.ldo + (int64_t)(head * a.group + first) * D, &so[0][0][0]);
    }
  }
  f += take;
  u += take;
  if (u == begin + units) {
    begin = u;
    if (++seq == a.batch) {
      seq = 0;
      ++column;
      begin = u = 0;
    }
  }
  if (f < fend) __syncthreads();  // the waves' sums have been read
  }
}

// The joins that the main kernel leaves, one workgroup per sequence and query
// head.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[256 * 6];
  const int lane = threadIdx.x & 63;
  const int cap = a.width * a.page_size, seq = blockIdx.x, qhead = blockIdx.y;
  const int units = units_of(seq_len(a.lens[seq], cap));
  if (units == 0) return;
  const Units un = count_units(a.lens, a.batch, cap, lane);
  int at = un.before;
  for (int i = un.i0; i < un.i1 && i < seq; ++i) at += units_of(seq_len(a.lens[i], cap));
  const int begin = __builtin_amdgcn_readlane(at, seq / un.per);
  const int head = qhead / a.group, qg = qhead % a.group;
  const int F = un.total * a.heads * a.qtiles;
  const Shares sh = make_shares(F, workgroups_of(F, a.workgroups));
  const int f0 = un.total * (head * a.qtiles + qg / 16) + begin;
  const int w0 = share_of(sh, f0), pieces = share_of(sh, f0 + units - 1) - w0 + 1;
  if (pieces == 1 || joined_here(pieces, min(16, a.group - qg / 16 * 16), D)) return;
  join_rows<T, D>(a, w0, pieces, qg % 16, 1, (T*)a.O + seq * a.ldo + (int64_t)qhead * D, lds);
}

template <typename T, bool FP8, int D>
hipError_t launch_decode(const DecodeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((decode_kernel<T, FP8, D>), dim3(a.workgroups), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  const int columns = a.heads * a.qtiles;
  const int64_t pieces = pieces_bound((int64_t)a.width * a.page_size, columns, a.workgroups);
  if (e != hipSuccess || joined_here((int)pieces, min(16, a.group), D)) return e;
  hipLaunchKernelGGL((join_kernel<T, D>), dim3(a.batch, a.heads * a.group), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// K and V beyond the L2s' 32 MiB are read past the caches (16 k tokens, 8 heads
// of 128: bf16 26.2 us against 31.4, f16 to E4M3 24.3 against 24.6; less is read
// faster through them, 2 heads of 64 8.1 against 8.6).  The cache is not
// written past them: the reader that follows pays for it (with it 39.4 us, 42.7
// that way, 43.4 with neither).
template <typename T, bool FP8, int D>
hipError_t launch_append(const AppendArgs& a, hipStream_t stream) {
  const dim3 grid((a.tokens + 3) / 4), block(256);
  if ((int64_t)a.tokens * a.heads * D * 4 > (int64_t)32 << 20)
    hipLaunchKernelGGL((append_kernel<T, FP8, D, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((append_kernel<T, FP8, D, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}
template <typename T, bool FP8>
hipError_t launch_append(const AppendArgs& a, int head_dim, hipStream_t stream) {
  return head_dim == 64 ? launch_append<T, FP8, 64>(a, stream) : launch_append<T, FP8, 128>(a, stream);
}

// ---------------------------------------------------------------------------
// argument checks
// ---------------------------------------------------------------------------
constexpr int64_t kLim = (int64_t)1 << 31;

gemm_epi_status check_cache(const gemm_epi_paged_cache* c, bool pointers) {
  if (!c || c->num_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0) return GEMM_EPI_ERR_INVALID_ARG;
  if (c->dtype != GEMM_EPI_F16 && c->dtype != GEMM_EPI_BF16 && c->dtype != GEMM_EPI_FP8_E4M3)
    return GEMM_EPI_ERR_INVALID_ARG;
  if (pointers) {
    const bool fp8 = c->dtype == GEMM_EPI_FP8_E4M3;
    if (!c->k || !c->v || fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr))
      return GEMM_EPI_ERR_INVALID_ARG;
  }
  if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size % 16 != 0 || c->page_size > 65536 || c->heads > 1024 ||
      c->num_pages >= kLim || c->num_pages * c->page_size >= kLim)
    return GEMM_EPI_ERR_UNSUPPORTED;
  if (pointers && (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 15u))
    return GEMM_EPI_ERR_UNSUPPORTED;
  return GEMM_EPI_OK;
}

gemm_epi_status check_sizes(int64_t page_size, int64_t batch, int64_t width) {
  if (batch < 0 || width <= 0) return GEMM_EPI_ERR_INVALID_ARG;
  // (positions and counts of units are 32-bit integers in the kernels)
  if (batch > 65535 || width >= kLim || width * page_size > kLim - 256 ||
      batch * ((width * page_size + kUnit - 1) / kUnit) >= kLim)
    return GEMM_EPI_ERR_UNSUPPORTED;
  return GEMM_EPI_OK;
}

gemm_epi_status check_table(const gemm_epi_paged_cache* c, const gemm_epi_page_table* t) {
  if (!t || t->ld < t->width) return GEMM_EPI_ERR_INVALID_ARG;
  const gemm_epi_status s = check_sizes(c->page_size, t->batch, t->width);
  if (s != GEMM_EPI_OK) return s;
  if (t->ld >= kLim) return GEMM_EPI_ERR_UNSUPPORTED;
  if (t->batch > 0 && (!t->pages || !t->lens || (((uintptr_t)t->pages | (uintptr_t)t->lens) & 3u)))
    return GEMM_EPI_ERR_INVALID_ARG;
  return GEMM_EPI_OK;
}

bool formats_fit(const gemm_epi_paged_cache* c, gemm_epi_dtype dtype) {
  return (dtype == GEMM_EPI_F16 || dtype == GEMM_EPI_BF16) && (c->dtype == dtype || c->dtype == GEMM_EPI_FP8_E4M3);
}

// Units of all columns of a full table.
int64_t units_bound(const gemm_epi_paged_cache* c, int64_t batch, int64_t width, int64_t q_heads) {
  return batch * ((width * c->page_size + kUnit - 1) / kUnit) * c->heads * ((q_heads / c->heads + 15) / 16);
}

struct Shape {
  int group, qtiles, workgroups;
};
Shape shape_of(const gemm_epi_paged_cache* c, int64_t batch, int64_t width, int64_t q_heads) {
  Shape s;
  s.group = (int)(q_heads / c->heads);
  s.qtiles = (s.group + 15) / 16;
  // no more workgroups than units
  const int64_t units = units_bound(c, batch, width, q_heads);
  const int most = workgroups_for((int)c->head_dim * (c->dtype == GEMM_EPI_FP8_E4M3 ? 1 : 2));
  s.workgroups = (int)(units < most ? units : most);
  return s;
}
size_t workspace_bytes(const gemm_epi_paged_cache* c, int64_t batch, int64_t width, int64_t q_heads) {
  return kWorkgroups * 4 + (size_t)shape_of(c, batch, width, q_heads).workgroups * 2 * (size_t)(16 * (c->head_dim + 2)) * 4;
}

template <typename T, bool FP8>
hipError_t launch_decode(const DecodeArgs& a, int head_dim, hipStream_t stream) {
  return head_dim == 64 ? launch_decode<T, FP8, 64>(a, stream) : launch_decode<T, FP8, 128>(a, stream);
}

}  // namespace paged
}  // namespace ge

extern "C" {

gemm_epi_status gemm_epi_cache_append(const gemm_epi_paged_cache* cache, const gemm_epi_page_table* table,
                                      const void* K, int64_t ldk, const void* V, int64_t ldv, const int32_t* starts,
                                      int64_t tokens, gemm_epi_dtype dtype, void* stream) {
  using namespace ge::paged;
  gemm_epi_status s = check_cache(cache, true);
  if (s == GEMM_EPI_OK) s = check_table(cache, table);
  if (s != GEMM_EPI_OK) return s;
  const int64_t row = cache->heads * cache->head_dim;
  if (!formats_fit(cache, dtype) || tokens < 0 || ldk < row || ldv < row || ((uintptr_t)starts & 3u) ||
      (!starts && tokens != table->batch))
    return GEMM_EPI_ERR_INVALID_ARG;
  // (four tokens a workgroup of 256: a grid holds below 2^32 threads)
  if (tokens > ((int64_t)1 << 26) - 4 || ldk % 8 != 0 || ldv % 8 != 0) return GEMM_EPI_ERR_UNSUPPORTED;
  if (tokens == 0 || table->batch == 0) return GEMM_EPI_OK;
  if (!K || !V) return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)K | (uintptr_t)V) & 15u) return GEMM_EPI_ERR_UNSUPPORTED;
  const AppendArgs a{(char*)cache->k, (char*)cache->v, cache->k_scale, cache->v_scale,
                     table->pages,    table->lens,     starts,         K,
                     V,               table->ld,       ldk,            ldv,
                     (int)cache->num_pages, (int)cache->page_size, (int)cache->heads, (int)table->width,
                     (int)table->batch, (int)tokens};
  const hipStream_t st = (hipStream_t)stream;
  const int d = (int)cache->head_dim;
  const bool fp8 = cache->dtype == GEMM_EPI_FP8_E4M3;
  const hipError_t e =
      dtype == GEMM_EPI_F16
          ? (fp8 ? launch_append<ge::f16, true>(a, d, st) : launch_append<ge::f16, false>(a, d, st))
          : (fp8 ? launch_append<ge::bf16, true>(a, d, st) : launch_append<ge::bf16, false>(a, d, st));
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}

size_t gemm_epi_attention_decode_workspace_size(const gemm_epi_paged_cache* cache, int64_t batch, int64_t width,
                                                int64_t q_heads) {
  using namespace ge::paged;
  if (check_cache(cache, false) != GEMM_EPI_OK || check_sizes(cache->page_size, batch, width) != GEMM_EPI_OK ||
      q_heads <= 0 || q_heads % cache->heads != 0 || q_heads > 16384 || batch == 0 ||
      units_bound(cache, batch, width, q_heads) >= kLim)
    return 0;
  return workspace_bytes(cache, batch, width, q_heads);
}

gemm_epi_status gemm_epi_attention_decode(const gemm_epi_paged_cache* cache, const gemm_epi_page_table* table,
                                          const void* Q, int64_t ldq, void* O, int64_t ldo, int64_t q_heads,
                                          gemm_epi_dtype dtype, void* workspace, size_t workspace_bytes_given,
                                          void* stream) {
  using namespace ge::paged;
  gemm_epi_status s = check_cache(cache, true);
  if (s == GEMM_EPI_OK) s = check_table(cache, table);
  if (s != GEMM_EPI_OK) return s;
  if (!formats_fit(cache, dtype) || q_heads <= 0 || q_heads % cache->heads != 0) return GEMM_EPI_ERR_INVALID_ARG;
  if (q_heads > 16384 || units_bound(cache, table->batch, table->width, q_heads) >= kLim)
    return GEMM_EPI_ERR_UNSUPPORTED;
  const int64_t row = q_heads * cache->head_dim;
  if (ldq < row || ldo < row) return GEMM_EPI_ERR_INVALID_ARG;
  if (ldq % 8 != 0 || ldo % 8 != 0) return GEMM_EPI_ERR_UNSUPPORTED;
  if (table->batch == 0) return GEMM_EPI_OK;
  if (!Q || !O || !workspace || workspace_bytes_given < workspace_bytes(cache, table->batch, table->width, q_heads))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)Q | (uintptr_t)O | (uintptr_t)workspace) & 15u) return GEMM_EPI_ERR_UNSUPPORTED;
  const Shape sh = shape_of(cache, table->batch, table->width, q_heads);
  const int d = (int)cache->head_dim;
  const DecodeArgs a{(const char*)cache->k,
                     (const char*)cache->v,
                     cache->k_scale,
                     cache->v_scale,
                     table->pages,
                     table->lens,
                     Q,
                     O,
                     (unsigned*)workspace,
                     (float*)((char*)workspace + kWorkgroups * 4),
                     table->ld,
                     ldq,
                     ldo,
                     (int)cache->num_pages,
                     (int)cache->page_size,
                     (int)cache->heads,
                     (int)table->width,
                     (int)table->batch,
                     sh.group,
                     sh.qtiles,
                     sh.workgroups,
                     make_divider((int)cache->page_size / 16),
                     (float)(1.4426950408889634 / __builtin_sqrt((double)d))};
  const hipStream_t st = (hipStream_t)stream;
  const bool fp8 = cache->dtype == GEMM_EPI_FP8_E4M3;
  const hipError_t e =
      dtype == GEMM_EPI_F16
          ? (fp8 ? launch_decode<ge::f16, true>(a, d, st) : launch_decode<ge::f16, false>(a, d, st))
          : (fp8 ? launch_decode<ge::bf16, true>(a, d, st) : launch_decode<ge::bf16, false>(a, d, st));
  if (e != hipSuccess) {
    ge::set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
  }
  return GEMM_EPI_OK;
}

}  // extern "C"
