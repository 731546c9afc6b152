// wave.hpp -- reductions over the 64 lanes of a wave without LDS: four DPP
// steps within rows of 16 lanes, then gfx950's v_permlane16_swap and
// v_permlane32_swap, which with the same value in both operands leave the
// even rows' (the lower half's) in one result and the odd rows' (the upper
// half's) in the other.
#pragma once

#include "common.hpp"

namespace ge {
namespace wave {

struct Sum {
  __device__ static __forceinline__ float op(float a, float b) { return a + b; }
};
struct Max {
  __device__ static __forceinline__ float op(float a, float b) { return fmaxf(a, b); }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// x combined over the four lanes l, l ^ 16, l ^ 32, l ^ 48.  (The results
// are copied first: a bit cast of a vector's element reads element 0.)
template <typename Op>
__device__ __forceinline__ float over_rows(float x) {
  const uint32_t a = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  const uint32_t b = __builtin_bit_cast(uint32_t, Op::op(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)));
  const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t s0 = s[0], s1 = s[1];
  return Op::op(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}

// x combined over the row of 16 lanes, the same bits in each of them.
template <typename Op>
__device__ __forceinline__ float over_row(float x) {
  x = Op::op(x, dpp<0xB1>(x));     // quad_perm [1, 0, 3, 2]
  x = Op::op(x, dpp<0x4E>(x));     // quad_perm [2, 3, 0, 1]
  x = Op::op(x, dpp<0x141>(x));    // row_half_mirror
  return Op::op(x, dpp<0x140>(x));  // row_mirror
}

// The largest x over the 8 or 16 lanes of a group.
template <int LANES>
__device__ __forceinline__ uint32_t max_over(uint32_t x) {
  static_assert(LANES == 8 || LANES == 16, "half a row or a row");
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true));
  if constexpr (LANES == 16) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, true));
  return x;
}

// x combined over the wave, the same bits in every lane.
template <typename Op>
__device__ __forceinline__ float all(float x) {
  return over_rows<Op>(over_row<Op>(x));
}

// The sum of x over this and all lower lanes (gfx9's scan by DPP: shifts
// within rows of 16, then the last lane of a row, and of the lower half,
// added to the rows above).
__device__ __forceinline__ int scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);  // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);  // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);  // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return x;
}

}  // namespace wave
}  // namespace ge
