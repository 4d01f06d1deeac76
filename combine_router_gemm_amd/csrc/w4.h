// 4-bit weights: E2M1 codes with one E8M0 scale byte per 32 k, packed in tiles (moe.h, "4-bit expert weights").
#pragma once

#include "common.h"
#include "../../include/moe.h"

namespace moe {

constexpr int W4_TILE_K = 128;    // k per code tile of 16 rows (1024 bytes)
constexpr int W4_STILE_K = 512;   // k per scale tile of 16 rows (256 bytes)
constexpr int W4_CODE_TILE = 1024;
constexpr int W4_SCALE_TILE = 256;

// The float32 2^(s - 127) of a scale byte (7 <= s <= 252)
__device__ __forceinline__ float w4_scale(uint32_t s) { return __uint_as_float(s << 23); }

// The eight codes of one 32-bit word times a scale as eight bf16 values, exact: v_cvt_scalef32_pk_bf16_fp4 takes
// one byte (two codes, the low half first) per instruction.
__device__ __forceinline__ u32x4 w4_to_bf16(uint32_t w, float scale) {
  u32x4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return v;
}
// the same as float32 values
__device__ __forceinline__ void w4_to_f32(uint32_t w, float scale, float (&o)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
  o[4] = c.x; o[5] = c.y; o[6] = d.x; o[7] = d.y;
}

}  // namespace moe
