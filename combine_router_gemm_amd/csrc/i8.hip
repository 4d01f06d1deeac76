// int8 rows of a matrix: codes and a scale per row from f32 or bf16 values, and back (moe.h, "int8 experts").
//
// Both are one pass over the data, bound by HBM. To quantise, a row's values stay in registers between its maximum and its
// codes, so it is read once: 16 or 64 lanes or a whole workgroup of 256 or 1024 take a row, as many as give each lane a few
// loads of 16 bytes. To expand, every load and store of a wave is one contiguous piece (with 16 codes per lane, whose values
// went out in stores 32 or 64 bytes apart, 8 x 4096 x 7168 to bf16 took 198 us).
#include <algorithm>

#include "common.h"
#include "i8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, const uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2, "codes of one 16-byte load");
  if constexpr (N == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
  else *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
}

// TPR threads per row, up to VPT 16-byte loads of each in registers; what a row has beyond them is read twice.
template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(TPR < kThreads ? kThreads : TPR) void quantize_i8_kernel(const T* __restrict__ w, int64_t rows,
                                                                                     int K, int8_t* __restrict__ codes,
                                                                                     float* __restrict__ scales) {
  constexpr int NTH = TPR < kThreads ? kThreads : TPR, VN = Vec<T>::N, RPB = NTH / TPR;
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
  constexpr int NTH = TPR < kThreads ? kThreads : TPR;
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
  else launch_quantize_t<T, 1024, 4>(p, rows, K, codes, scales, stream);
}

// A thread's VN codes make one 16-byte store; U of them, a workgroup's width apart.
template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_i8_kernel(const int8_t* __restrict__ codes,
                                                                const float* __restrict__ scales, int64_t vecs,
                                                                int per_row, T* __restrict__ w) {
  constexpr int VN = Vec<T>::N, U = 4, STEP = kThreads * U;
  for (int64_t base = (int64_t)blockIdx.x * STEP; base < vecs; base += (int64_t)gridDim.x * STEP) {
    const int64_t row0 = base / per_row;  // uniform: the row of a thread is a 32-bit division from there
    const unsigned rest = (unsigned)(base - row0 * per_row);
    u32x2 c[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = base + u * kThreads + threadIdx.x;
      const bool in = at < vecs;
      if constexpr (VN == 8) c[u] = in ? *reinterpret_cast<const u32x2*>(codes + at * VN) : u32x2{0u, 0u};
      else c[u] = u32x2{in ? *reinterpret_cast<const uint32_t*>(codes + at * VN) : 0u, 0u};
      sc[u] = in ? scales[row0 + (rest + u * kThreads + threadIdx.x) / (unsigned)per_row] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = base + u * kThreads + threadIdx.x;
      float f[VN];
#pragma unroll
      for (int q = 0; q < VN; ++q) f[q] = (float)(int8_t)(c[u][q / 4] >> (8 * (q % 4))) * sc[u];
      if (at < vecs) st16_nt(w + at * VN, pack(f));
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
  const int vn = bf16 ? 8 : 4;
  const int64_t vecs = rows * (K / vn);
  const int grid = (int)std::min<int64_t>(ceil_div_host64(vecs, kThreads * 4), 1 << 22);
  if (bf16)
    dequantize_i8_kernel<bf16_t><<<grid, kThreads, 0, stream>>>(codes, scales, vecs, K / vn, static_cast<bf16_t*>(w));
  else dequantize_i8_kernel<float><<<grid, kThreads, 0, stream>>>(codes, scales, vecs, K / vn, static_cast<float*>(w));
  return hipGetLastError();
}

}  // namespace moe
