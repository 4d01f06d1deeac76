// int8 rows of a matrix: codes and a scale per row from f32 or bf16 values, and back (moe.h, "int8 experts").
//
// Both are one pass over the data, bound by HBM. To quantise, a row's values stay in registers between its maximum and its
// codes, so it is read once: 16 or 64 lanes or a whole workgroup take a row, as many as give each lane a few loads of
// 16 bytes.
#include <algorithm>

#include "common.h"
#include "i8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int NTH = 256;

template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, const uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2, "codes of one 16-byte load");
  if constexpr (N == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
  else *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
}

// TPR threads per row, up to VPT 16-byte loads of each in registers; what a row has beyond them is read twice.
template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(NTH) void quantize_i8_kernel(const T* __restrict__ w, int64_t rows, int K,
                                                         int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int VN = Vec<T>::N, RPB = NTH / TPR;
  __shared__ uint32_t s_top[NTH / 64];
  const int tid = threadIdx.x, lane = tid % TPR;
  const int nvec = K / VN;
  for (int64_t b = blockIdx.x; b * RPB < rows; b += gridDim.x) {
    const int64_t row = b * RPB + tid / TPR;
    const bool on = row < rows;
    const T* src = w + (on ? row : 0) * K;
    u32x4 raw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * TPR + lane;
      raw[i] = on && v < nvec ? ld16_nt(src + (int64_t)v * VN) : u32x4{0u, 0u, 0u, 0u};
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[VN];
      unpack(raw[i], f);
      top = abs_top(f, top);
    }
    if (on)
      for (int v = VPT * TPR + lane; v < nvec; v += TPR) {
        float f[VN];
        unpack(ld16(src + (int64_t)v * VN), f);
        top = abs_top(f, top);
      }
#pragma unroll
    for (int off = min(TPR, 64) / 2; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if constexpr (TPR > 64) {
      __syncthreads();  // the previous row's maxima have been read
      if ((tid & 63) == 0) s_top[tid >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NTH / 64; ++i) top = max(top, s_top[i]);
    }
    if (!on) continue;  // no barrier follows for TPR <= 64, and a whole workgroup shares `on` otherwise
    const I8Row r = i8_row(top);
    int8_t* dst = codes + row * K;
    if (lane == 0) scales[row] = r.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * TPR + lane;
      if (v < nvec) {
        float f[VN];
        uint32_t c[VN / 4];
        unpack(raw[i], f);
        i8_codes(f, r, c);
        store_codes(dst + (int64_t)v * VN, c);
      }
    }
    for (int v = VPT * TPR + lane; v < nvec; v += TPR) {
      float f[VN];
      uint32_t c[VN / 4];
      unpack(ld16(src + (int64_t)v * VN), f);
      i8_codes(f, r, c);
      store_codes(dst + (int64_t)v * VN, c);
    }
  }
}

template <typename T, int TPR, int VPT>
void launch_quantize_t(const T* w, int64_t rows, int K, int8_t* codes, float* scales, hipStream_t stream) {
  const int64_t blocks = ceil_div_host64(rows, NTH / TPR);
  quantize_i8_kernel<T, TPR, VPT><<<(int)std::min<int64_t>(blocks, 1 << 20), NTH, 0, stream>>>(w, rows, K, codes, scales);
}

template <typename T>
void launch_quantize(const void* w, int64_t rows, int K, int8_t* codes, float* scales, hipStream_t stream) {
  const T* p = static_cast<const T*>(w);
  const int nvec = K / Vec<T>::N;
  if (nvec <= 32) launch_quantize_t<T, 16, 2>(p, rows, K, codes, scales, stream);
  else if (nvec <= 256) launch_quantize_t<T, 64, 4>(p, rows, K, codes, scales, stream);
  else if (nvec <= 1024) launch_quantize_t<T, 256, 4>(p, rows, K, codes, scales, stream);
  else launch_quantize_t<T, 256, 16>(p, rows, K, codes, scales, stream);
}

// 16 codes per thread: one 16-byte load, two or four 16-byte stores.
template <typename T>
__global__ __launch_bounds__(NTH) void dequantize_i8_kernel(const int8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, int64_t chunks,
                                                           int per_row, T* __restrict__ w) {
  for (int64_t base = (int64_t)blockIdx.x * NTH; base < chunks; base += (int64_t)gridDim.x * NTH) {
    const int64_t at = base + threadIdx.x;
    if (at >= chunks) return;
    const int64_t row0 = base / per_row;  // uniform: the row of a thread is a 32-bit division from there
    const int64_t row = row0 + ((unsigned)(base - row0 * per_row) + threadIdx.x) / (unsigned)per_row;
    const float sc = scales[row];
    const u32x4 c = ld16_nt(codes + at * 16);
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) f[4 * i + q] = (float)(int8_t)(c[i] >> (8 * q)) * sc;
    constexpr int VN = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 16 / VN; ++i) {
      float o[VN];
#pragma unroll
      for (int q = 0; q < VN; ++q) o[q] = f[i * VN + q];
      st16_nt(w + at * 16 + i * VN, pack(o));
    }
  }
}

}  // namespace

hipError_t launch_quantize_i8(const void* w, int bf16, int64_t rows, int K, int8_t* codes, float* scales,
                              hipStream_t stream) {
  if (bf16) launch_quantize<bf16_t>(w, rows, K, codes, scales, stream);
  else launch_quantize<float>(w, rows, K, codes, scales, stream);
  return hipGetLastError();
}

hipError_t launch_dequantize_i8(const int8_t* codes, const float* scales, int64_t rows, int K, void* w, int bf16,
                                hipStream_t stream) {
  const int64_t chunks = rows * (K / 16);
  const int grid = (int)std::min<int64_t>(ceil_div_host64(chunks, NTH), 1 << 22);
  if (bf16)
    dequantize_i8_kernel<bf16_t><<<grid, NTH, 0, stream>>>(codes, scales, chunks, K / 16, static_cast<bf16_t*>(w));
  else dequantize_i8_kernel<float><<<grid, NTH, 0, stream>>>(codes, scales, chunks, K / 16, static_cast<float*>(w));
  return hipGetLastError();
}

}  // namespace moe
