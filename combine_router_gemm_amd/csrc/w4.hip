// 4-bit expert weights: quantisation to E2M1 codes with group scales, and back (moe.h, "4-bit expert weights").
//
// Both kernels are one pass over the data, bound by HBM: 2 (bf16) or 4 (f32) bytes of a weight against 17/32 of
// a byte of its code and scale. A workgroup handles 16 rows x 512 k: four code tiles that are contiguous in
// memory (4 KB) and one scale tile (256 bytes). A wave takes whole rows, each lane eight consecutive k (16 bytes
// of bf16), so the weight side moves in contiguous kilobytes; four lanes share a group, whose maximum they
// exchange by DPP. The tile order of the codes is made in LDS, so the packed side is contiguous as well.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "w4.h"

namespace moe {

namespace {

constexpr int W4_ROWS = 16;
constexpr int W4_NTH = 256;
constexpr int W4_RPW = W4_ROWS / (W4_NTH / 64);  // rows per wave

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float (&v)[8]) {
  unpack(ld16_nt(p), v);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  unpack(ld16_nt(p), *reinterpret_cast<float(*)[4]>(&v[0]));
  unpack(ld16_nt(p + 4), *reinterpret_cast<float(*)[4]>(&v[4]));
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false)));
  return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false)));
}

// The smallest E with a <= 6 * 2^E, clamped: a = m 2^e with 1 <= m < 2, and 6 * 2^E = 1.5 * 2^(E + 2), so E is
// e - 2 for m <= 1.5 and e - 1 above. A subnormal a has e = -127 here and lands on the lower clamp either way.
__device__ __forceinline__ int group_exponent(float a) {
  if (a == 0.f) return 0;
  const uint32_t b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 127;
  const int E = (b & 0x7fffffu) <= 0x400000u ? e - 2 : e - 1;
  return min(125, max(-120, E));
}

// The E2M1 codes of eight values over 2^E, the first in the low four bits: v_cvt_scalef32_pk_fp4_f32 divides by the
// scale, rounds to nearest with ties to the even code, clamps to +-6 and keeps the sign of zero, two values per
// instruction. Counting the seven borders below each value by comparisons instead took 136-155 us against 91 for
// 8 x 4096 x 7168 bf16 weights: 20 operations a weight made the vector units the bound.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&v)[8], int E) {
  const float scale = __uint_as_float((uint32_t)(127 + E) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}

template <typename T>
__global__ __launch_bounds__(W4_NTH) void quantize_w4_kernel(const T* __restrict__ w, int64_t blocks, int K,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) uint32_t s_codes[4 * W4_CODE_TILE / 4];
  __shared__ __attribute__((aligned(16))) uint8_t s_scales[W4_SCALE_TILE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kc = (K + W4_TILE_K - 1) / W4_TILE_K, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t rb = b / ks;
    const int kb = (int)(b - rb * ks);
    const int k = kb * W4_STILE_K + lane * 8;
    const bool in = k < K;  // a group is wholly inside or past K (K % 32 == 0)
    float v[W4_RPW][8];
#pragma unroll
    for (int i = 0; i < W4_RPW; ++i) {
      const int64_t row = rb * W4_ROWS + wave * W4_RPW + i;
      load8(w + row * K + (in ? k : 0), v[i]);
    }
    const int g = lane >> 2;  // group inside the 512 k: tile g / 4, quarter g % 4
#pragma unroll
    for (int i = 0; i < W4_RPW; ++i) {
      float a = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) a = fmaxf(a, fabsf(v[i][q]));
      a = quad_max(in ? a : 0.f);
      const int E = group_exponent(a);
      const uint32_t word = e2m1_codes(v[i], E);
      const int r = wave * W4_RPW + i;
      const int own = r + 16 * (g & 3);  // the tile lane that owns this group
      s_codes[(g >> 2) * (W4_CODE_TILE / 4) + own * 4 + (lane & 3)] = in ? word : 0u;
      if ((lane & 3) == 0) s_scales[own * 4 + (g >> 2)] = (uint8_t)(E + 127);
    }
    __syncthreads();
    if (kb * 4 + (tid >> 6) < kc)
      st16(codes + (rb * kc + kb * 4) * W4_CODE_TILE + tid * 16, *reinterpret_cast<const u32x4*>(s_codes + tid * 4));
    if (tid < W4_SCALE_TILE / 16)
      st16(scales + (rb * ks + kb) * W4_SCALE_TILE + tid * 16, *reinterpret_cast<const u32x4*>(s_scales + tid * 16));
    __syncthreads();
  }
}

__device__ __forceinline__ void store8(bf16_t* p, uint32_t word, float sc) { st16_nt(p, w4_to_bf16(word, sc)); }
__device__ __forceinline__ void store8(float* p, uint32_t word, float sc) {
  float o[8];
  w4_to_f32(word, sc, o);
  const float lo[4] = {o[0], o[1], o[2], o[3]}, hi[4] = {o[4], o[5], o[6], o[7]};
  st16_nt(p, pack(lo));
  st16_nt(p + 4, pack(hi));
}

template <typename T>
__global__ __launch_bounds__(W4_NTH) void dequantize_w4_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t blocks,
                                                              int K, T* __restrict__ w) {
  __shared__ __attribute__((aligned(16))) uint32_t s_codes[4 * W4_CODE_TILE / 4];
  __shared__ __attribute__((aligned(16))) uint8_t s_scales[W4_SCALE_TILE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kc = (K + W4_TILE_K - 1) / W4_TILE_K, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t rb = b / ks;
    const int kb = (int)(b - rb * ks);
    if (kb * 4 + (tid >> 6) < kc)
      *reinterpret_cast<u32x4*>(s_codes + tid * 4) = ld16_nt(codes + (rb * kc + kb * 4) * W4_CODE_TILE + tid * 16);
    if (tid < W4_SCALE_TILE / 16)
      *reinterpret_cast<u32x4*>(s_scales + tid * 16) = ld16_nt(scales + (rb * ks + kb) * W4_SCALE_TILE + tid * 16);
    __syncthreads();
    const int k = kb * W4_STILE_K + lane * 8, g = lane >> 2;
    if (k < K) {
#pragma unroll
      for (int i = 0; i < W4_RPW; ++i) {
        const int r = wave * W4_RPW + i;
        const int own = r + 16 * (g & 3);
        store8(w + (rb * W4_ROWS + r) * K + k, s_codes[(g >> 2) * (W4_CODE_TILE / 4) + own * 4 + (lane & 3)],
               w4_scale(s_scales[own * 4 + (g >> 2)]));
      }
    }
    __syncthreads();
  }
}

int w4_grid(int64_t blocks) { return (int)std::min<int64_t>(blocks, 1 << 20); }

}  // namespace

hipError_t launch_quantize_w4(const void* w, int bf16, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
  const int64_t blocks = rows / W4_ROWS * ceil_div_host(K, W4_STILE_K);
  if (bf16)
    quantize_w4_kernel<bf16_t><<<w4_grid(blocks), W4_NTH, 0, stream>>>(static_cast<const bf16_t*>(w), blocks, K,
                                                                       codes, scales);
  else
    quantize_w4_kernel<float><<<w4_grid(blocks), W4_NTH, 0, stream>>>(static_cast<const float*>(w), blocks, K, codes,
                                                                      scales);
  return hipGetLastError();
}

hipError_t launch_dequantize_w4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, void* w, int bf16,
                                hipStream_t stream) {
  const int64_t blocks = rows / W4_ROWS * ceil_div_host(K, W4_STILE_K);
  if (bf16)
    dequantize_w4_kernel<bf16_t><<<w4_grid(blocks), W4_NTH, 0, stream>>>(codes, scales, blocks, K,
                                                                         static_cast<bf16_t*>(w));
  else
    dequantize_w4_kernel<float><<<w4_grid(blocks), W4_NTH, 0, stream>>>(codes, scales, blocks, K,
                                                                        static_cast<float*>(w));
  return hipGetLastError();
}

}  // namespace moe
