// Gradients of the combine (moe_combine_backward) and of the router (moe_route_backward).
//
// combine: y[t] = sum_j w[t, j] out[row(t, j)] over kept slots, so d_w[t, j] = dy[t] . out[row] and d_out[row] = w[t, j] dy[t].
//   One workgroup per token reads dy[t] once and its rows once. Bound: HBM.
//
// router: w = softmax over the selected logits, logits = x Wr^T + b. With c_j = w_j (d_w_j - sum_i w_i d_w_i), the gradient of
//   the logits is d_in plus c_j at the selected experts; then d_x = d_logits Wr, d_Wr = d_logits^T x, d_b = the column sums.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "mfma.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int NTH = 256;

// VPT 16-byte slices of dy per thread stay in registers; what a longer row has beyond them is read again for each slot.
template <typename T, int VPT>
__global__ __launch_bounds__(NTH) void combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ out_buf,
                                                              const int* __restrict__ pair_row,
                                                              const float* __restrict__ topk_w, int H, int k,
                                                              float* __restrict__ d_w, T* __restrict__ d_out) {
  constexpr int VN = Vec<T>::N;
  __shared__ float s_sum[MOE_MAX_TOPK][NTH / 64];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int nvec = H / VN;
  const T* g = dy + t * H;
  u32x4 raw[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * NTH;
    raw[i] = v < nvec ? ld16(g + (int64_t)v * VN) : u32x4{0u, 0u, 0u, 0u};
  }
  for (int j = 0; j < k; ++j) {
    const int row = pair_row[t * k + j];
    if (row < 0) continue;
    const float w = topk_w[t * k + j];
    const T* src = out_buf + (int64_t)row * H;
    T* dst = d_out ? d_out + (int64_t)row * H : nullptr;
    float acc = 0.f;
    auto slice = [&](u32x4 gv, u32x4 ov, int v) {
      float a[VN], b[VN];
      unpack(gv, a);
      unpack(ov, b);
#pragma unroll
      for (int q = 0; q < VN; ++q) acc = fmaf(a[q], b[q], acc);
      if (dst) {
#pragma unroll
        for (int q = 0; q < VN; ++q) a[q] *= w;
        st16_nt(dst + (int64_t)v * VN, pack(a));
      }
    };
    u32x4 o[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * NTH;
      if (v < nvec) o[i] = ld16_nt(src + (int64_t)v * VN);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * NTH;
      if (v < nvec) slice(raw[i], o[i], v);
    }
    for (int v = tid + VPT * NTH; v < nvec; v += NTH) slice(ld16(g + (int64_t)v * VN), ld16_nt(src + (int64_t)v * VN), v);
    const float sum = wave_sum(acc);
    if ((tid & 63) == 0) s_sum[j][tid >> 6] = sum;
  }
  __syncthreads();
  if (tid < k) {
    float v = 0.f;
    if (pair_row[t * k + tid] >= 0)
      for (int i = 0; i < NTH / 64; ++i) v += s_sum[tid][i];
    d_w[t * k + tid] = v;
  }
}

// ---- router ----

// One wave per token: d_in's row, with c_j added at the selected experts (an id given twice gets both).
__global__ __launch_bounds__(NTH) void route_dlogits_kernel(const int* __restrict__ ids, const float* __restrict__ w,
                                                           const float* __restrict__ d_w, const float* d_in, int T_,
                                                           int E, int k, float* d_logits) {
  const int64_t t = (int64_t)blockIdx.x * (NTH / 64) + (threadIdx.x >> 6);
  if (t >= T_) return;
  const int lane = lane_id();
  float wj = 0.f, dj = 0.f;
  int id = -1;
  if (d_w && lane < k) {
    wj = w[t * k + lane];
    dj = d_w[t * k + lane];
    id = ids[t * k + lane];
  }
  const float c = wj * (dj - wave_sum(wj * dj));
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    float v = d_in && e < E ? d_in[t * E + e] : 0.f;
    if (d_w)
      for (int j = 0; j < k; ++j) {
        const float cj = __shfl(c, j, 64);  // every lane takes part in both exchanges
        v += __shfl(id, j, 64) == e ? cj : 0.f;
      }
    if (e < E) d_logits[t * E + e] = v;
  }
}

// C[m, n] = sum_k A(m, k) B[k, n] in fp32 on v_mfma_f32_32x32x2_f32, B's rows contiguous in n. TRANS: A(m, k) = A[k, m], else
// A[m, k]. 64 x 64 tiles, four waves of 32 x 32, K in steps of 16 through LDS.
template <typename TB, typename TO, bool TRANS>
__global__ __launch_bounds__(NTH) void route_grad_gemm_kernel(const float* __restrict__ A, const TB* __restrict__ B, int M,
                                                             int N, int K, int lda, TO* __restrict__ C) {
  constexpr int BM = 64, BN = 64, BK = 16, PAD = 4;
  __shared__ float s_a[BK][BM + PAD], s_b[BK][BN + PAD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x16 acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  for (int k0 = 0; k0 < K; k0 += BK) {
    __syncthreads();
    for (int i = tid; i < BK * BM; i += NTH) {
      const int kk = TRANS ? i / BM : i % BK, mm = TRANS ? i % BM : i / BK;
      const bool in = k0 + kk < K && m0 + mm < M;
      s_a[kk][mm] = !in ? 0.f : TRANS ? A[(int64_t)(k0 + kk) * lda + m0 + mm] : A[(int64_t)(m0 + mm) * lda + k0 + kk];
    }
    for (int i = tid; i < BK * BN; i += NTH) {
      const int kk = i / BN, nn = i % BN;
      s_b[kk][nn] = k0 + kk < K && n0 + nn < N ? to_f32(B[(int64_t)(k0 + kk) * N + n0 + nn]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; kk += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(s_a[kk + (lane >> 5)][wm + (lane & 31)],
                                                 s_b[kk + (lane >> 5)][wn + (lane & 31)], acc, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int m = m0 + wm + Op32::out_row(lane, q), n = n0 + wn + (lane & 31);
    if (m < M && n < N) C[(int64_t)m * N + n] = from_f32<TO>(acc[q]);
  }
}

// Column sums of d_logits [T, E]: a workgroup per 64 columns, its waves' partial sums added in their order.
__global__ __launch_bounds__(1024) void route_dbias_kernel(const float* __restrict__ d, int T_, int E, float* __restrict__ out) {
  __shared__ double s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  double v = 0.0;
  if (e < E)
    for (int64_t t = wave; t < T_; t += 16) v += (double)d[t * E + e];
  s[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && e < E) {
    v = 0.0;
    for (int i = 0; i < 16; ++i) v += s[i][lane];
    out[e] = (float)v;
  }
}

}  // namespace

hipError_t launch_combine_backward(const void* dy, int bf16, const void* out_buf, const moe_layout_t& L,
                                   const float* topk_w, float* d_w, void* d_out, hipStream_t stream) {
  const int nvec = L.H / (bf16 ? 8 : 4);
#define MOE_GO(TY, VPT)                                                                                            \
  combine_backward_kernel<TY, VPT><<<L.T, NTH, 0, stream>>>(static_cast<const TY*>(dy), static_cast<const TY*>(out_buf), \
                                                            L.pair_row, topk_w, L.H, L.k, d_w, static_cast<TY*>(d_out))
  if (bf16) {
    if (nvec <= NTH) MOE_GO(bf16_t, 1);
    else if (nvec <= 2 * NTH) MOE_GO(bf16_t, 2);
    else MOE_GO(bf16_t, 4);
  } else {
    if (nvec <= NTH) MOE_GO(float, 1);
    else if (nvec <= 2 * NTH) MOE_GO(float, 2);
    else MOE_GO(float, 4);
  }
#undef MOE_GO
  return hipGetLastError();
}

size_t route_backward_workspace_bytes(int T, int H, int E, int bf16) {
  (void)T, (void)H, (void)E, (void)bf16;
  return 0;
}

hipError_t launch_route_backward(const RouteBackward& r, hipStream_t stream) {
  if (r.T > 0) {
    route_dlogits_kernel<<<ceil_div_host(r.T, NTH / 64), NTH, 0, stream>>>(r.ids, r.w, r.d_w, r.d_in, r.T, r.E, r.k,
                                                                          r.d_logits);
    if (r.d_x) {
      const dim3 g(ceil_div_host(r.H, 64), ceil_div_host(r.T, 64));
      if (r.bf16)
        route_grad_gemm_kernel<float, bf16_t, false><<<g, NTH, 0, stream>>>(r.d_logits, r.w_router, r.T, r.H, r.E, r.E,
                                                                           static_cast<bf16_t*>(r.d_x));
      else
        route_grad_gemm_kernel<float, float, false><<<g, NTH, 0, stream>>>(r.d_logits, r.w_router, r.T, r.H, r.E, r.E,
                                                                          static_cast<float*>(r.d_x));
    }
  }
  if (r.d_w_router) {
    const dim3 g(ceil_div_host(r.H, 64), ceil_div_host(r.E, 64));
    if (r.bf16)
      route_grad_gemm_kernel<bf16_t, float, true><<<g, NTH, 0, stream>>>(r.d_logits, static_cast<const bf16_t*>(r.x), r.E,
                                                                        r.H, r.T, r.E, r.d_w_router);
    else
      route_grad_gemm_kernel<float, float, true><<<g, NTH, 0, stream>>>(r.d_logits, static_cast<const float*>(r.x), r.E,
                                                                       r.H, r.T, r.E, r.d_w_router);
  }
  if (r.d_bias) route_dbias_kernel<<<ceil_div_host(r.E, 64), 1024, 0, stream>>>(r.d_logits, r.T, r.E, r.d_bias);
  return hipGetLastError();
}

}  // namespace moe
