// Wave-level reductions and the integer sort key of a logit, shared by the router's top-k kernels and the
// few-token layer.
#pragma once

#include "common.h"

namespace moe {

// Maximum of x over the 64 lanes of the wave, in every lane: DPP swaps within quads, 8- and 16-lane
// mirrors (VALU operations, no LDS), then the four row maxima read into scalar registers.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_f32<0xB1>(x));   // quad_perm [1, 0, 3, 2]
  x = fmaxf(x, dpp_f32<0x4E>(x));   // quad_perm [2, 3, 0, 1]
  x = fmaxf(x, dpp_f32<0x141>(x));  // row_half_mirror
  x = fmaxf(x, dpp_f32<0x140>(x));  // row_mirror
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 48));
  return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}
// Sum of x over the 64 lanes of the wave, in every lane, in a fixed order: pairs, quads, 8- and 16-lane
// groups by DPP (each partner adds the same two values, so every lane of a row holds the same bits),
// then (row 0 + row 1) + (row 2 + row 3).
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_f32<0xB1>(x);
  x += dpp_f32<0x4E>(x);
  x += dpp_f32<0x141>(x);
  x += dpp_f32<0x140>(x);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 48));
  return (r0 + r1) + (r2 + r3);
}

// Integer max over the 64 lanes of the wave, in every lane (same DPP pattern as wave_max; v_max_i32 needs
// no NaN handling).
template <int CTRL>
__device__ __forceinline__ int dpp_i32(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ int wave_max_i32(int x) {
  x = max(x, dpp_i32<0xB1>(x));   // quad_perm [1, 0, 3, 2]
  x = max(x, dpp_i32<0x4E>(x));   // quad_perm [2, 3, 0, 1]
  x = max(x, dpp_i32<0x141>(x));  // row_half_mirror
  x = max(x, dpp_i32<0x140>(x));  // row_mirror
  const int r0 = __builtin_amdgcn_readlane(x, 0), r1 = __builtin_amdgcn_readlane(x, 16);
  const int r2 = __builtin_amdgcn_readlane(x, 32), r3 = __builtin_amdgcn_readlane(x, 48);
  return max(max(r0, r1), max(r2, r3));
}
// Order-preserving integer key of a float that is not NaN and not -0: a larger float has a larger key,
// equal floats have equal keys, and key_float inverts it.
__device__ __forceinline__ int float_key(float v) {
  const int b = __float_as_int(v);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float key_float(int key) { return __int_as_float(key >= 0 ? key : key ^ 0x7fffffff); }

}  // namespace moe
