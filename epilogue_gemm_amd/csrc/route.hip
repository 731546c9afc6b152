// route.hip -- the router of a layer of experts: the k largest logits of each
// token and their weights, and the entries (token, choice) in the stable order
// of their experts.
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

// The larger of two keys, by their bits.
struct MaxBits {
  __device__ static __forceinline__ float op(float a, float b) {
    return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)));
  }
};

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

// A wave a token, V consecutive experts a lane.
template <typename T, int V>
__global__ __launch_bounds__(256) void route_kernel(Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.ldl;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    key[i] = e < a.experts ? key_of((float)row[e]) : 0u;
  }
  float top = 0.0f, all = 0.0f, sum = 0.0f, w = 0.0f;
  int id = -1;
  for (int j = 0; j < a.per; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) best = key[i], at = i;
    const uint32_t m = __builtin_bit_cast(uint32_t, wave::all<MaxBits>(__builtin_bit_cast(float, best)));
    if (m == 0) break;
    const int src = __builtin_ctzll(__builtin_amdgcn_ballot_w64(best == m));
    const int e = __builtin_amdgcn_readlane(lane * V + at, src);
    const float x = logit_of(m);
    if (j == 0) {
      top = x;
      if (!a.sigmoid && !a.renormalise) {
        // (infinities share the softmax)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] != 0) all += key[i] == m ? 1.0f : exp_of(logit_of(key[i]) - top);
        all = wave::all<wave::Sum>(all);
      }
    }
    float p;
    if (!a.sigmoid) p = x == top ? 1.0f : exp_of(x - top);
    // (divided by the largest where that may be too small for fp32)
    else if (a.renormalise && top < 0.0f) p = exp_of(x - top) * (1.0f + exp_of(top)) / (1.0f + exp_of(x));
    else p = 1.0f / (1.0f + exp_of(-x));
    sum += p;
    if (lane == j) id = e, w = p;
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = 0;
    }
  }
  if (lane < a.per) {
    const float over = a.renormalise ? sum : a.sigmoid ? 1.0f : all;
    a.ids[t * a.per + lane] = id;
    a.weights[t * a.per + lane] = id < 0 ? 0.0f : w / over * a.scale;
  }
}

// ---------------------------------------------------------------------------
// the entries by group
// ---------------------------------------------------------------------------
struct GroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order;
  int rows, groups;
};

// A workgroup a group (the last one: the entries of none).  Each reads all
// ids twice: to count those of lower groups and of its own, a wave for each
// sixteenth of them, then to write its own in their order.
__global__ __launch_bounds__(1024) void group_kernel(GroupArgs a) {
  __shared__ int below[16], own[16];
  const int g = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t part = ((int64_t)a.rows + 1023) / 1024 * 64, i0 = part * wave, i1 = std::min<int64_t>(a.rows, i0 + part);
  auto group = [&](int64_t i) __attribute__((always_inline)) {
    const uint32_t id = i < i1 ? (uint32_t)a.ids[i] : ~0u;
    return id < (uint32_t)a.groups ? (int)id : i < i1 ? a.groups : a.groups + 1;
  };
  int lower = 0, mine = 0;
  for (int64_t i = i0; i < i1; i += 64) {
    const int x = group(i + lane);
    lower += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x < g));
    mine += __builtin_popcountll(__builtin_amdgcn_ballot_w64(x == g));
  }
  if (lane == 0) below[wave] = lower, own[wave] = mine;
  __syncthreads();
  int at = 0;
  for (int i = 0; i < 16; ++i) at += below[i];
  if (threadIdx.x == 0) a.offsets[g] = at;
  for (int i = 0; i < wave; ++i) at += own[i];
  for (int64_t i = i0; i < i1; i += 64) {
    const bool is = group(i + lane) == g;
    const uint64_t which = __builtin_amdgcn_ballot_w64(is);
    if (is) {
      const int to = at + __builtin_popcountll(which & (((uint64_t)1 << lane) - 1));
      a.order[to] = g < a.groups ? (int)(i + lane) : -1;
    }
    at += __builtin_popcountll(which);
  }
}

hipError_t launch_group(const GroupArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(group_kernel, dim3(a.groups + 1), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_route(const Args& a, hipStream_t stream) {
  const dim3 grid((uint32_t)(((int64_t)a.tokens + 3) / 4)), block(256);
  if (a.experts <= 64) hipLaunchKernelGGL((route_kernel<T, 1>), grid, block, 0, stream, a);
  else if (a.experts <= 128) hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, 0, stream, a);
  else if (a.experts <= 256) hipLaunchKernelGGL((route_kernel<T, 4>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, 0, stream, a);
  return hipGetLastError();
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
  hipError_t e = hipSuccess;
  if (tokens > 0)
    e = dtype == GEMM_EPI_F32 ? launch_route<float>(a, st)
                              : dtype == GEMM_EPI_F16 ? launch_route<ge::f16>(a, st) : launch_route<ge::bf16>(a, st);
  if (e == hipSuccess && offsets)
    e = launch_group(GroupArgs{ids, offsets, order, (int)(tokens * per), (int)experts}, st);
  return status_of(e);
}

}  // extern "C"
