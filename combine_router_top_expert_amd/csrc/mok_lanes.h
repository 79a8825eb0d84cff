// Butterfly reductions over groups of L consecutive lanes (L a power of two
// up to 64), without LDS traffic.  Step 1 and 2 exchange inside a quad
// (quad_perm); steps 4 and 8 read the mirrored lane of the half row and of
// the row, which holds the same value as the xor partner because the lanes
// of a quad (of a half row) already agree; steps 16 and 32 swap rows and
// halves of the wave (v_permlane16_swap, v_permlane32_swap).  Every lane of
// the group ends with the same bits: the two operands of a step are only
// exchanged, and the operations commute.
#pragma once

#include "mok_common.h"

namespace mok {

template <int CTRL>
__device__ __forceinline__ float dpp_f(float x) {
  return __uint_as_float((unsigned)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xF, 0xF, true));
}

struct OpAdd {
  __device__ __forceinline__ static float op(float a, float b) { return a + b; }
};
struct OpMax {
  __device__ __forceinline__ static float op(float a, float b) { return __builtin_fmaxf(a, b); }
};

template <int L, class Op>
__device__ __forceinline__ float group_reduce(float x) {
  if constexpr (L >= 2) x = Op::op(x, dpp_f<0xB1>(x));
  if constexpr (L >= 4) x = Op::op(x, dpp_f<0x4E>(x));
  if constexpr (L >= 8) x = Op::op(x, dpp_f<0x141>(x));
  if constexpr (L >= 16) x = Op::op(x, dpp_f<0x140>(x));
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = Op::op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = Op::op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return x;
}

}  // namespace mok
