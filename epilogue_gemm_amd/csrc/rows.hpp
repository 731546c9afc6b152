// rows.hpp -- eight consecutive values of a row, for the kernels that pass once
// over rows of any length and alignment.
#pragma once

#include "common.hpp"

namespace ge {
namespace rows {

// Eight consecutive values of a row, the last ones of it perhaps fewer (zeros
// then).  ANY: rows at any address of an element (a 16-byte access off its
// alignment is one instruction all the same) and of any length; else whole
// and aligned.  PAST: read past the caches.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
template <bool ANY, bool PAST = false>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int j, int cols) {
  if (j >= cols) return u32x4{};
  if constexpr (!ANY && PAST) return __builtin_nontemporal_load((const u32x4*)(row + j));
  if constexpr (!ANY) return *(const u32x4*)(row + j);
  if (j + 8 <= cols) return *(const u32x4_any*)(row + j);
  uint32_t v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = j + u < cols ? row[j + u] : 0u;
  return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}
template <typename T>
__device__ __forceinline__ void widen(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = to_f32(__builtin_bit_cast(T, (uint16_t)(w[i] & 0xffffu)));
    f[2 * i + 1] = to_f32(__builtin_bit_cast(T, (uint16_t)(w[i] >> 16)));
  }
}
template <typename T, bool ANY>
__device__ __forceinline__ void store8(T* row, int j, int cols, const float (&f)[8]) {
  if (j >= cols) return;
  if (ANY && j + 8 > cols) {
    for (int u = 0; u < 8; ++u)
      if (j + u < cols) row[j + u] = from_f32<T>(f[u]);
    return;
  }
  if constexpr (sizeof(T) == 1) {
    // within +-448 but for the last place of fp32, by the scale: the
    // conversion rounds that back, no clamp needed
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    const u32x2 w = {(uint32_t)lo, (uint32_t)hi};
    if constexpr (ANY) *(u32x2_any*)(row + j) = w;
    else *(u32x2*)(row + j) = w;
  } else {
    const u32x4 w = {pack2_out<T>(f[0], f[1]), pack2_out<T>(f[2], f[3]), pack2_out<T>(f[4], f[5]), pack2_out<T>(f[6], f[7])};
    if constexpr (ANY) *(u32x4_any*)(row + j) = w;
    else *(u32x4*)(row + j) = w;
  }
}

}  // namespace rows
}  // namespace ge
