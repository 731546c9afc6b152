// route.hip -- the router of a layer of experts: the k largest logits of each
// token and their weights, and the entries (token, choice) in the stable order
// of their experts.  A choice is a largest key over lanes and its removal; bound by
// these instructions for many tokens (16384 tokens, 8 of 256: bf16 6.9 us, f32 8.3;
// 64 lanes a token 12.4 and 14.6), by launches and latencies for few (32 tokens, 8
// of 128, with the order 4.7 us in one kernel, in two 7).
#include <algorithm>

#include "kernels.hpp"
#include "wave.hpp"

#include "../../include/gemm_epi_experts.h"

namespace ge {
namespace route {

constexpr float kNegInf = -__builtin_inff();

struct Args {
  const void* logits;
  int32_t* ids;
  float* weights;
  int64_t ldl;
  int tokens, experts, per;
  int sigmoid, renormalise;
  float scale;
};

// exp(x): the product with log2 e in two parts, as its rounding alone would
// cost |x| half steps.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float hi = 1.44269502e+00f, lo = 1.92596304e-08f;  // log2 e
  const float p = x * hi, r = __builtin_fmaf(x, hi, -p) + x * lo;
  // (at an infinity of p, r is none)
  return x < -200.0f ? 0.0f : x > 200.0f ? __builtin_inff() : __builtin_amdgcn_exp2f(p) * __builtin_fmaf(r, 0.693147181f, 1.0f);
}

// Whole numbers over the L lanes of a token (16 or 64), the same in each.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int L, typename Op>
__device__ __forceinline__ uint32_t over(uint32_t x, Op&& op) {
  x = op(x, dpp<0xB1>(x));   // quad_perm [1, 0, 3, 2]
  x = op(x, dpp<0x4E>(x));   // quad_perm [2, 3, 0, 1]
  x = op(x, dpp<0x141>(x));  // row_half_mirror
  x = op(x, dpp<0x140>(x));  // row_mirror
  if constexpr (L == 64) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const uint32_t r0 = r[0], r1 = r[1], y = op(r0, r1);
    const auto s = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    x = op(s0, s1);
  }
  return x;
}
template <int L>
__device__ __forceinline__ float sum_over(float x) {
  return L == 64 ? wave::all<wave::Sum>(x) : wave::over_row<wave::Sum>(x);
}

// A logit as an unsigned integer in the same order, never 0 but for minus
// infinity and NaN, which are not chosen.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > kNegInf)) return 0;
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // (-0 and 0 are equal)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
// Of a 16-bit format the key has the expert too, a lower one above: the order of
// the 16-bit patterns in the upper half.
template <typename T>
__device__ __forceinline__ uint32_t key_of(T x, int e) {
  const uint32_t k = key_of((float)x);
  if constexpr (sizeof(T) == 4) return k;
  else {
    const uint32_t h = bits16((T)((float)x + 0.0f)), o = h & 0x8000u ? ~h & 0xffffu : h | 0x8000u;
    return k == 0 ? 0u : o << 16 | (0xffffu - e);
  }
}
template <typename T>
__device__ __forceinline__ float logit_of(uint32_t key) {
  if constexpr (sizeof(T) == 4) return logit_of(key);
  else {
    const uint32_t o = key >> 16;
    return (float)__builtin_bit_cast(T, (uint16_t)(o & 0x8000u ? o & 0x7fffu : ~o));
  }
}

// L lanes a token, V consecutive experts a lane: for each choice the largest key,
// the lowest expert that has it, and that one taken out.  Lane j % L then holds
// choice j, and writes it (to `out` too, which is then not null, in LDS).
template <typename T, int V, int L>
__device__ __forceinline__ void route_token(const Args& a, int64_t t, int lane, int* out) {
  const T* row = (const T*)a.logits + t * a.ldl;
  uint32_t key[V];
  struct __attribute__((packed, aligned(sizeof(T)))) Lane {
    T x[V];
  };
  if ((lane + 1) * V <= a.experts) {
    const Lane l = *(const Lane*)(row + lane * V);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key_of<T>(l.x[i], lane * V + i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      key[i] = e < a.experts ? key_of<T>(row[e], e) : 0u;
    }
  }
  constexpr int KEPT = 64 / L;  // choices a lane holds (64 at most)
  uint32_t chosen[KEPT] = {};
  int id[KEPT];
  float all = 0.0f;
  uint32_t first = 0;
  for (int j = 0; j < a.per; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, key[i]);
    m = over<L>(m, [](uint32_t x, uint32_t y) { return max(x, y); });
    if (j == 0) {
      first = m;
      if (!a.sigmoid && !a.renormalise) {
        // (infinities share the softmax)
        const float top = logit_of<T>(m);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = logit_of<T>(key[i]);
          if (key[i] != 0) all += x == top ? 1.0f : exp_of(x - top);
        }
        all = sum_over<L>(all);
      }
    }
    if (L == 64 && m == 0) break;  // (of several tokens a wave, others may go on)
    uint32_t e;
    if constexpr (sizeof(T) == 2) {
      e = 0xffffu - (m & 0xffffu);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] == m ? 0u : key[i];
    } else {
      e = ~0u;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) e = key[i] == m ? (uint32_t)(lane * V + i) : e;
      e = over<L>(e, [](uint32_t x, uint32_t y) { return min(x, y); });
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = (uint32_t)(lane * V + i) == e ? 0u : key[i];
    }
#pragma unroll
    for (int s = 0; s < KEPT; ++s)
      if (lane + L * s == j) id[s] = (int)e, chosen[s] = m;
  }
  const float top = logit_of<T>(first);
  float w[KEPT], sum = 0.0f;
#pragma unroll
  for (int s = 0; s < KEPT; ++s) {
    const float x = logit_of<T>(chosen[s]);
    if (chosen[s] == 0) w[s] = 0.0f;
    else if (!a.sigmoid) w[s] = x == top ? 1.0f : exp_of(x - top);
    // (divided by the largest where that may be too small for fp32)
    else if (a.renormalise && top < 0.0f) w[s] = exp_of(x - top) * (1.0f + exp_of(top)) / (1.0f + exp_of(x));
    else w[s] = 1.0f / (1.0f + exp_of(-x));
    sum += w[s];
  }
  if (a.renormalise) sum = sum_over<L>(sum);
  const float whole = a.renormalise ? sum : a.sigmoid ? 1.0f : all;
#pragma unroll
  for (int s = 0; s < KEPT; ++s)
    if (lane + L * s < a.per) {
      const int64_t q = t * a.per + lane + L * s;
      const int e = chosen[s] == 0 ? -1 : id[s];
      a.ids[q] = e;
      a.weights[q] = e < 0 ? 0.0f : w[s] / whole * a.scale;
      if (out) out[q] = e;
    }
}

template <typename T, int V, int L>
__global__ __launch_bounds__(256) void route_kernel(Args a) {
  const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (t < a.tokens) route_token<T, V, L>(a, t, threadIdx.x % L, nullptr);
}

// ---------------------------------------------------------------------------
// the entries by group
// ---------------------------------------------------------------------------
struct GroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order;
  int rows, groups;
};

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(4)));

// A workgroup a group.  Each reads all ids to count those of lower groups, in
// rounds of a batch of 2048 consecutive ones a wave, a lane four of each 256, and
// keeps a bit for each of its own (KEPT: up to 131072 entries, else it reads them
// again); then it writes these in their order.  Bound by the comparisons, five
// instructions for each id and group (131072 ids of 256 groups 11.2 us; with a
// scan over lanes for each 256 ids 20.7).
constexpr int kKept = 131072;
template <bool KEPT>
__global__ __launch_bounds__(1024) void group_kernel(GroupArgs a) {
  __shared__ int below[16], own[4][16];
  const int g = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rounds = (int)(((int64_t)a.rows + 32767) / 32768);
  // Four of this lane's ids: those of lower groups (an id of none is above all
  // groups as an unsigned number), and a bit for each of its own, the first one
  // the highest: a comparison and an addition with carry each.
  auto four = [&](const i32x4& x, uint32_t& bits, uint32_t& lower) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      lower += (uint32_t)x[u] < (uint32_t)g;
      bits = bits + bits + (x[u] == g);
    }
  };
  uint32_t lower = 0;
  // this wave's batch of a round: its own ones' bits
  auto batch = [&](int round) __attribute__((always_inline)) {
    const int64_t i0 = (int64_t)round * 32768 + 2048 * wave;
    uint32_t bits = 0;
    if (i0 >= a.rows) return bits;
    const int32_t* p = a.ids + i0 + 4 * lane;
    i32x4 x[8];
    if (i0 + 2048 <= a.rows) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = *(const i32x4_any*)(p + 256 * j);
#pragma unroll
      for (int j = 0; j < 8; ++j) four(x[j], bits, lower);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[j][u] = i0 + 256 * j + 4 * lane + u < a.rows ? p[256 * j + u] : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j) four(x[j], bits, lower);
    }
    return bits;
  };
  // this wave's own ones of a batch, from place `to` on: each block's counts in
  // 16 bits of four words, summed over lower lanes and lower blocks, are the
  // places, of which a lane takes one after the other
  auto write = [&](int round, uint32_t bits, int to) __attribute__((always_inline)) {
    uint32_t place[4];
    int before = to;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __builtin_popcount(bits >> (28 - 8 * i) & 15u), hi = __builtin_popcount(bits >> (24 - 8 * i) & 15u);
      const uint32_t n = lo | hi << 16, upto = (uint32_t)wave::scan((int)n), sum = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
      const int mid = before - to + (int)(sum & 0xffffu);
      place[i] = upto - n + ((uint32_t)(before - to) | (uint32_t)mid << 16);
      before = to + mid + (int)(sum >> 16);
    }
    const int first = round * 32768 + 2048 * wave + 4 * lane;
    while (__builtin_amdgcn_ballot_w64(bits != 0)) {
      if (bits != 0) {
        const int b = __builtin_clz(bits), j = b >> 2, half = (j & 1) * 16;
        uint32_t p = place[0];
        p = j >> 1 == 1 ? place[1] : p;
        p = j >> 1 == 2 ? place[2] : p;
        p = j >> 1 == 3 ? place[3] : p;
#pragma unroll
        for (int i = 0; i < 4; ++i) place[i] += j >> 1 == i ? 1u << half : 0u;
        a.order[to + (int)(p >> half & 0xffffu)] = first + 256 * j + (b & 3);
        bits &= ~(0x80000000u >> b);
      }
    }
  };
  uint32_t kept[4] = {};
  if constexpr (KEPT) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < rounds) kept[k] = batch(k);
  } else {
    for (int k = 0; k < rounds; ++k) batch(k);
  }
  const int lower_sum = wave::scan((int)lower);
  if (lane == 63) below[wave] = lower_sum;
  if constexpr (KEPT) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = wave::scan(__builtin_popcount(kept[k]));
      if (lane == 63) own[k][wave] = n;
    }
  }
  __syncthreads();
  int at = 0;
  for (int i = 0; i < 16; ++i) at += below[i];
  if (threadIdx.x == 0) a.offsets[g] = at;
  if constexpr (KEPT) {
    const int n = (&own[0][0])[lane], upto = at + wave::scan(n);
    at = __builtin_amdgcn_readlane(upto, 63);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < rounds) write(k, kept[k], __builtin_amdgcn_readlane(upto - n, 16 * k + wave));
  } else {
    for (int k = 0; k < rounds; ++k) {
      // (a wave a round ahead writes the other half)
      const uint32_t bits = batch(k);
      const int n = wave::scan(__builtin_popcount(bits));
      if (lane == 63) own[k & 1][wave] = n;
      __syncthreads();
      int to = at;
      for (int i = 0; i < 16; ++i) {
        to += i < wave ? own[k & 1][i] : 0;
        at += own[k & 1][i];
      }
      write(k, bits, to);
    }
  }
  // the last group's workgroup knows where the order ends
  if (g == a.groups - 1) {
    if (threadIdx.x == 0) a.offsets[a.groups] = at;
    for (int64_t i = at + (int64_t)threadIdx.x; i < a.rows; i += 1024) a.order[i] = -1;
  }
}

// Router and order of few entries by one workgroup: 16 lanes a token; then, as no
// token has an expert twice, a bit for each token in a mask for each expert, whose
// counts give the offsets and whose lower bits an entry's place.
constexpr int kFew = 512, kFewTokens = 64, kFewExperts = 256;
template <typename T, int V>
__global__ __launch_bounds__(1024) void route_few(Args a, GroupArgs b) {
  __shared__ int ids[kFew], begin[kFewExperts + 1], part[4];
  __shared__ uint32_t mask[kFewExperts][2];
  const int i = threadIdx.x, lane = i & 63;
  if (i < 2 * kFewExperts) (&mask[0][0])[i] = 0;
  if (i / 16 < a.tokens) route_token<T, V, 16>(a, i / 16, i % 16, ids);
  __syncthreads();
  const int id = i < b.rows ? ids[i] : -1, t = i / a.per;
  if (id >= 0) atomicOr(&mask[id][t >> 5], 1u << (t & 31));
  __syncthreads();
  int incl = 0, n = 0;
  if (i < kFewExperts) {
    n = __builtin_popcount(mask[i][0]) + __builtin_popcount(mask[i][1]);
    incl = wave::scan(n);
    if (lane == 63) part[i >> 6] = incl;
  }
  __syncthreads();
  if (i < kFewExperts) {
    for (int w = 0; w < i >> 6; ++w) incl += part[w];
    begin[i + 1] = incl;
    if (i == 0) begin[0] = 0;
    if (i < b.groups) b.offsets[i] = incl - n;
    if (i == b.groups - 1) b.offsets[b.groups] = incl;
  }
  __syncthreads();
  if (id >= 0) {
    const uint32_t lo = mask[id][0], hi = mask[id][1], under = (1u << (t & 31)) - 1;
    b.order[begin[id] + (t < 32 ? __builtin_popcount(lo & under) : __builtin_popcount(lo) + __builtin_popcount(hi & under))] = i;
  }
  if (i < b.rows && i >= begin[kFewExperts]) b.order[i] = -1;
}

hipError_t launch_group(const GroupArgs& a, hipStream_t stream) {
  if (a.rows <= kKept) hipLaunchKernelGGL(group_kernel<true>, dim3(a.groups), dim3(1024), 0, stream, a);
  else hipLaunchKernelGGL(group_kernel<false>, dim3(a.groups), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

template <typename T, int V, int L>
hipError_t launch_tokens(const Args& a, hipStream_t stream) {
  constexpr int n = 256 / L;
  hipLaunchKernelGGL((route_kernel<T, V, L>), dim3((uint32_t)(((int64_t)a.tokens + n - 1) / n)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_few(const Args& a, const GroupArgs& b, hipStream_t stream) {
  hipLaunchKernelGGL((route_few<T, V>), dim3(1), dim3(1024), 0, stream, a, b);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_route(const Args& a, const GroupArgs* b, hipStream_t stream) {
  if (b && a.tokens <= kFewTokens && b->rows <= kFew && a.experts <= kFewExperts) {
    if (a.experts <= 16) return launch_few<T, 1>(a, *b, stream);
    if (a.experts <= 64) return launch_few<T, 4>(a, *b, stream);
    if (a.experts <= 128) return launch_few<T, 8>(a, *b, stream);
    return launch_few<T, 16>(a, *b, stream);
  }
  hipError_t e;
  if (a.experts > 512) e = launch_tokens<T, 16, 64>(a, stream);
  else if (a.experts > 384) e = launch_tokens<T, 32, 16>(a, stream);
  else if (a.experts > 256) e = launch_tokens<T, 24, 16>(a, stream);
  else if (a.experts > 128) e = launch_tokens<T, 16, 16>(a, stream);
  else if (a.experts > 64) e = launch_tokens<T, 8, 16>(a, stream);
  else if (a.experts > 16) e = launch_tokens<T, 4, 16>(a, stream);
  else e = launch_tokens<T, 1, 16>(a, stream);
  return e != hipSuccess || !b ? e : launch_group(*b, stream);
}

constexpr int64_t kLim = (int64_t)1 << 31;
constexpr int64_t kMaxTokens = (int64_t)1 << 25;  // four a workgroup of 256: a grid holds below 2^32 threads

gemm_epi_status status_of(hipError_t e) {
  if (e == hipSuccess) return GEMM_EPI_OK;
  set_last_hip_error((int)e);
  return GEMM_EPI_ERR_HIP;
}

}  // namespace route
}  // namespace ge

extern "C" {

gemm_epi_status gemm_epi_group_rows(const int32_t* ids, int64_t rows, int64_t groups, int32_t* offsets, int32_t* order,
                                    void* stream) {
  using namespace ge::route;
  if (rows < 0 || groups <= 0 || !offsets || (rows > 0 && (!ids || !order)) ||
      (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)order) & 3u))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (groups > 1024 || rows >= kLim) return GEMM_EPI_ERR_UNSUPPORTED;
  return status_of(launch_group(GroupArgs{ids, offsets, order, (int)rows, (int)groups}, (hipStream_t)stream));
}

gemm_epi_status gemm_epi_route(const void* logits, int64_t ldl, gemm_epi_dtype dtype, int64_t tokens, int64_t experts,
                               int64_t per, gemm_epi_score score, int renormalise, float scale, int32_t* ids,
                               float* weights, int32_t* offsets, int32_t* order, void* stream) {
  using namespace ge::route;
  if (dtype != GEMM_EPI_F32 && dtype != GEMM_EPI_F16 && dtype != GEMM_EPI_BF16) return GEMM_EPI_ERR_INVALID_ARG;
  if (score != GEMM_EPI_SOFTMAX && score != GEMM_EPI_SIGMOID) return GEMM_EPI_ERR_INVALID_ARG;
  if (tokens < 0 || experts <= 0 || per <= 0 || per > experts || ldl < experts ||
      !(__builtin_fabsf(scale) < __builtin_inff()))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (tokens > 0 && (!logits || !ids || !weights)) return GEMM_EPI_ERR_INVALID_ARG;
  // (without tokens an order has no elements, and may have no address)
  if (offsets ? tokens > 0 && !order : order != nullptr) return GEMM_EPI_ERR_INVALID_ARG;
  if (((uintptr_t)logits & (dtype == GEMM_EPI_F32 ? 3u : 1u)) ||
      (((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)offsets | (uintptr_t)order) & 3u))
    return GEMM_EPI_ERR_INVALID_ARG;
  if (experts > 1024 || per > 64 || tokens > kMaxTokens || tokens * per >= kLim || ldl >= kLim) return GEMM_EPI_ERR_UNSUPPORTED;
  const hipStream_t st = (hipStream_t)stream;
  const Args a{logits, ids, weights, ldl, (int)tokens, (int)experts, (int)per, (int)score, renormalise != 0, scale};
  const GroupArgs b{ids, offsets, order, (int)(tokens * per), (int)experts}, *grouped = offsets ? &b : nullptr;
  hipError_t e = hipSuccess;
  if (tokens == 0) e = offsets ? launch_group(b, st) : e;
  else if (dtype == GEMM_EPI_F32) e = launch_route<float>(a, grouped, st);
  else e = dtype == GEMM_EPI_F16 ? launch_route<ge::f16>(a, grouped, st) : launch_route<ge::bf16>(a, grouped, st);
  return status_of(e);
}

}  // extern "C"
