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

template <int L>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (L >= 2) x = x + dpp_f<0xB1>(x);
  if constexpr (L >= 4) x = x + dpp_f<0x4E>(x);
  if constexpr (L >= 8) x = x + dpp_f<0x141>(x);
  if constexpr (L >= 16) x = x + dpp_f<0x140>(x);
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// fp32 values as signed integers of the same order (-0 below +0; a positive
// NaN above infinity, a negative one below -inf), so that a maximum is one
// integer instruction with the exchange folded in.
__device__ __forceinline__ int float_order(float x) {
  const int b = (int)__float_as_uint(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_float(int o) { return __uint_as_float((unsigned)(o ^ ((o >> 31) & 0x7FFFFFFF))); }

template <int CTRL>
__device__ __forceinline__ int dpp_i(int x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, true);
}
template <int L>
__device__ __forceinline__ int group_max(int x) {
  if constexpr (L >= 2) x = max(x, dpp_i<0xB1>(x));
  if constexpr (L >= 4) x = max(x, dpp_i<0x4E>(x));
  if constexpr (L >= 8) x = max(x, dpp_i<0x141>(x));
  if constexpr (L >= 16) x = max(x, dpp_i<0x140>(x));
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap((unsigned)x, (unsigned)x, false, false);
    x = max((int)r[0], (int)r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap((unsigned)x, (unsigned)x, false, false);
    x = max((int)r[0], (int)r[1]);
  }
  return x;
}

}  // namespace mok
