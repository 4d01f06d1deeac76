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
// Three products share one operand, the gradient of the logits, of T x E values: small, but the factor of 2 T E H operations
// with either matrix. bf16 layers run them on bf16 MFMA, whose products are exact in fp32, with the fp32 operands cut into
// bf16 parts of 8 bits: d_w_router (fp32) takes d_logits in three parts, which hold all of it, and x as it is; d_x, rounded to
// bf16 in the end, takes d_logits and the weight in two parts each (16 bits) and three of their four products. fp32 layers run
// on fp32 MFMA.
//   route_grad_prep   d_logits, its column sums per 32 tokens, and the parts, laid out as the matrix unit takes them: a
//                     fragment (32 rows x 16 k) is the 1 KB that a wave loads at once, lane l row l % 32, k = 8 (l / 32) on.
//                     The transposes are made here, where they cost little.
//   route_dx          the weight's parts of 64 or 128 columns stay in LDS while the tokens stream past.
//   route_dw          x is transposed on its way to LDS: a thread loads 8 x 8 values and puts pairs of rows together.
constexpr int kRows = 32, kStep = 16, kFrag = 1024;  // rows and k of a fragment, its bytes
constexpr int kPairCols = 64;  // columns of x that two fragments of the weight hold, the even ones and the odd ones

struct GradArgs {
  RouteBackward r;
  int tb, ek, eb, hb;    // 32-token blocks, 16-expert steps, 32-expert blocks, 64-column blocks
  unsigned char* px;     // [tb][ek][2 parts] fragments: rows tokens, k experts
  unsigned char* pw;     // [eb][2 tb][3 parts] fragments: rows experts, k tokens
  unsigned char* wt;     // [hb][ek][2 columns parities][2 parts] fragments: rows columns of x, k experts
  float* bias_part;      // [tb][E]
  float* partial;        // [splits][E][H]
  int splits, chunks_per_split;
};

// Eight values as N bf16 parts, each the nearest bf16 of what the parts before it leave.
template <int N>
__device__ __forceinline__ void store_parts(float (&v)[8], unsigned char* frag, int lane) {
#pragma unroll
  for (int p = 0; p < N; ++p) {
    st16(frag + p * kFrag + lane * 16, pack(v));
    if (p + 1 < N) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = bf16_rest(v[q]);
    }
  }
}

// Workgroups [0, tb): 32 tokens each. The others: 64 columns x 32 experts of the weight each.
__global__ __launch_bounds__(NTH) void route_grad_prep_kernel(GradArgs a) {
  constexpr int PITCH = MOE_MAX_EXPERTS + 1;
  __shared__ float s[kRows * PITCH];
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, E = r.E, k = r.k;
  if ((int)blockIdx.x < a.tb) {
    const int64_t t0 = (int64_t)blockIdx.x * kRows;
    const int n = (int)min((int64_t)kRows, r.T - t0);
    const int ep = a.eb * kRows;  // experts with the padding of a fragment, zeros
    for (int i = tid >> 6; i < kRows; i += NTH / 64)
      for (int e = tid & 63; e < ep; e += 64) s[i * PITCH + e] = r.d_in && i < n && e < E ? r.d_in[(t0 + i) * E + e] : 0.f;
    __syncthreads();
    if (r.d_w && tid < n) {  // a thread per token, so that an id given twice gets both
      const int64_t at = (t0 + tid) * k;
      float w[MOE_MAX_TOPK], d[MOE_MAX_TOPK], sum = 0.f;
      int id[MOE_MAX_TOPK];
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOPK; ++j) {
        w[j] = j < k ? r.w[at + j] : 0.f;
        d[j] = j < k ? r.d_w[at + j] : 0.f;
        id[j] = j < k ? r.ids[at + j] : -1;
      }
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOPK; ++j)
        if (j < k) sum = fmaf(w[j], d[j], sum);
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOPK; ++j)
        if (id[j] >= 0 && id[j] < E) s[tid * PITCH + id[j]] += w[j] * (d[j] - sum);
    }
    __syncthreads();
    for (int i = tid >> 6; i < n; i += NTH / 64)
      for (int e = tid & 63; e < E; e += 64) r.d_logits[(t0 + i) * E + e] = s[i * PITCH + e];
    if (r.d_bias)
      for (int e = tid; e < E; e += NTH) {
        float v = 0.f;
        for (int i = 0; i < n; ++i) v += s[i * PITCH + e];
        a.bias_part[(int64_t)blockIdx.x * E + e] = v;
      }
    if (a.px)
      for (int i = tid; i < a.ek * 64; i += NTH) {
        const int lane = i & 63, step = i >> 6;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = s[(lane & 31) * PITCH + step * kStep + (lane >> 5) * 8 + q];
        store_parts<2>(v, a.px + ((int64_t)blockIdx.x * a.ek + step) * 2 * kFrag, lane);
      }
    if (a.pw)
      for (int i = tid; i < a.eb * 2 * 64; i += NTH) {
        const int lane = i & 63, half = (i >> 6) & 1, b = i >> 7;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = s[(half * kStep + (lane >> 5) * 8 + q) * PITCH + b * kRows + (lane & 31)];
        store_parts<3>(v, a.pw + ((int64_t)b * a.tb * 2 + (int64_t)blockIdx.x * 2 + half) * 3 * kFrag, lane);
      }
    return;
  }
  constexpr int WP = kPairCols + 4;
  const int i = blockIdx.x - a.tb, b = i / a.eb, e0 = i % a.eb * kRows, h0 = b * kPairCols;
  for (int v = tid; v < kRows * kPairCols / 4; v += NTH) {
    const int e = v / (kPairCols / 4), c = v % (kPairCols / 4) * 4;
    const bool in = e0 + e < E && h0 + c < r.H;
    *reinterpret_cast<u32x4*>(s + e * WP + c) = in ? ld16(r.w_router + (int64_t)(e0 + e) * r.H + h0 + c) : u32x4{0u, 0u, 0u, 0u};
  }
  __syncthreads();
  const int lane = tid & 63, odd = (tid >> 6) & 1, step = tid >> 7;
  if (e0 / kStep + step < a.ek) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = s[(step * kStep + (lane >> 5) * 8 + q) * WP + 2 * (lane & 31) + odd];
    store_parts<2>(v, a.wt + (((int64_t)b * a.ek + e0 / kStep + step) * 2 + odd) * 2 * kFrag, lane);
  }
}

// d_x: a wave computes 64 tokens x 64 columns, WT x WH waves. The columns' parts are in LDS for good; the tokens' fragments come
// from memory one step ahead, across the ends of the token tiles.
template <int WT, int WH>
__global__ __launch_bounds__(WT * WH * 64) void route_dx_kernel(GradArgs a) {
  constexpr int NT = WT * WH * 64;
  extern __shared__ __attribute__((aligned(1024))) unsigned char s_w[];
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wh = wave % WH, wt = wave / WH;
  const int b0 = blockIdx.x * WH;
  const int per_block = a.ek * 4 * kFrag;  // bytes of a 64-column block
  for (int i = tid * 16; i < min(WH, a.hb - b0) * per_block; i += NT * 16) st16(s_w + i, ld16(a.wt + (int64_t)b0 * per_block + i));
  __syncthreads();
  if (b0 + wh >= a.hb) return;
  const unsigned char* w = s_w + wh * per_block + lane * 16;
  const int tiles = (a.tb + 2 * WT - 1) / (2 * WT);  // of 64 WT tokens
  u32x4 fa[2][2][2];  // buffer, 32-token block, part
  auto load = [&](int tile, int step, u32x4 (&f)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tb = min((tile * WT + wt) * 2 + i, a.tb - 1);
#pragma unroll
      for (int p = 0; p < 2; ++p) f[i][p] = ld16(a.px + (((int64_t)tb * a.ek + step) * 2 + p) * kFrag + lane * 16);
    }
  };
  f32x16 acc[2][2];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  };
  clear();
  int tile = blockIdx.y, step = 0;
  if (tile < tiles) load(tile, 0, fa[0]);
  auto one = [&](u32x4 (&now)[2][2], u32x4 (&next)[2][2]) {
    const int nstep = step + 1 < a.ek ? step + 1 : 0, ntile = nstep ? tile : tile + (int)gridDim.y;
    if (ntile < tiles) load(ntile, nstep, next);
    u32x4 fb[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) fb[j][p] = ld16(w + ((step * 2 + j) * 2 + p) * kFrag);
#pragma unroll
    for (int pp = 2; pp >= 0; --pp) {  // second parts first
      const int pa = pp == 1, pb = pp == 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x4 x[1] = {now[i][pa]}, y[1] = {fb[j][pb]};
          Op32::step(acc[i][j], x, y);
        }
    }
    if (nstep == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int64_t t = (int64_t)((tile * WT + wt) * 2 + i) * kRows + Op32::out_row(lane, q);
          const int h = (b0 + wh) * kPairCols + 2 * (lane & 31);
          if (t < r.T && h < r.H)
            *reinterpret_cast<uint32_t*>(static_cast<bf16_t*>(r.d_x) + t * r.H + h) = pack2_bf16(acc[i][0][q], acc[i][1][q]);
        }
      clear();
    }
    tile = ntile;
    step = nstep;
  };
  while (tile < tiles) {
    one(fa[0], fa[1]);
    if (tile < tiles) one(fa[1], fa[0]);
  }
}

// Column sums of d_logits from those of 32 tokens: 64 columns per workgroup of eight waves, their sums added in order.
__device__ __forceinline__ void bias_sums(const GradArgs& a, int block, double* s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = block * 64 + lane;
  double v = 0.0;
  if (e < a.r.E)
    for (int i = wave; i < a.tb; i += 8) v += (double)a.bias_part[(int64_t)i * a.r.E + e];
  s[wave * 64 + lane] = v;
  __syncthreads();
  if (wave == 0 && e < a.r.E) {
    v = 0.0;
    for (int i = 0; i < 8; ++i) v += s[i * 64 + lane];
    a.r.d_bias[e] = (float)v;
  }
}
__global__ __launch_bounds__(512) void route_dbias_kernel(GradArgs a) {
  __shared__ double s[512];
  bias_sums(a, blockIdx.x, s);
}

// d_w_router: eight waves, WE along the experts (32 each) and 8 / WE along the tokens, whose sums are added in the end; 128
// columns of x. Tokens go in chunks of 256: a thread loads 8 tokens x 8 columns of the next chunk while this one is multiplied.
// In LDS the chunk is fragments [16 steps][4 column blocks]; in a fragment the 16 bytes of column c are at place
// c ^ (its group of 8 in the 128 columns), so that the writes of a wave, at a stride of 8 columns, touch all banks.
// Workgroups past the column tiles add up the bias.
constexpr int kDwCols = 128, kDwChunk = 256;
template <int WE>
__global__ __launch_bounds__(512) void route_dw_kernel(GradArgs a, int col_tiles) {
  constexpr int KW = 8 / WE, CHUNK = kDwChunk * kDwCols * 2;
  extern __shared__ __attribute__((aligned(1024))) unsigned char s_x[];  // two chunks
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, lane = tid & 63;
  if ((int)blockIdx.x >= col_tiles) {
    if (blockIdx.y == 0 && blockIdx.z == 0) bias_sums(a, blockIdx.x - col_tiles, reinterpret_cast<double*>(s_x));
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int we = wave % WE, kw = wave / WE;
  const int eb = blockIdx.z * 8 + we;  // this wave's 32 experts
  const int h0 = blockIdx.x * kDwCols;
  const int steps = a.tb * 2, chunks = (steps + 15) / 16;
  const int c0 = blockIdx.y * a.chunks_per_split, c1 = min(chunks, c0 + a.chunks_per_split);
  const bf16_t* x = static_cast<const bf16_t*>(r.x);
  const int g8 = tid & 15, t8 = tid >> 4;  // this thread's 8 columns and 8 tokens of a chunk
  const bool in_h = h0 + g8 * 8 < r.H;
  u32x4 raw[8];
  auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = (int64_t)c * kDwChunk + t8 * 8 + i;
      raw[i] = in_h && t < r.T ? ld16_nt(x + t * r.H + h0 + g8 * 8) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  auto store = [&](int slot) {
    unsigned char* base = s_x + slot * CHUNK + (((t8 >> 1) * 4 + (g8 >> 2)) * 64 + (t8 & 1) * 32 + (g8 & 3) * 8) * 16;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      u32x4 v;
#pragma unroll
      for (int p = 0; p < 4; ++p)  // tokens 2 p and 2 p + 1 of column c
        v[p] = __builtin_amdgcn_perm(raw[2 * p + 1][c >> 1], raw[2 * p][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
      st16(base + ((c ^ g8) & 7) * 16, v);
    }
  };
  f32x16 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[j][q] = 0.f;
  const unsigned char* pw = a.pw + (int64_t)min(eb, a.eb - 1) * steps * 3 * kFrag + lane * 16;
  int rd[4];  // this lane's column in the four blocks
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = j * 4 + ((lane & 31) >> 3);
    rd[j] = (j * 64 + (lane & 32) + (lane & 24) + ((lane ^ g) & 7)) * 16;
  }
  if (c0 < c1) {
    load(c0);
    store(0);
  }
  for (int c = c0; c < c1; ++c) {
    lds_barrier();  // chunk c is in LDS, and chunk c - 1 has been read
    if (c + 1 < c1) load(c + 1);
    const unsigned char* base = s_x + ((c - c0) & 1) * CHUNK;
    const int s_end = min(16, steps - c * 16);
    u32x4 fa[2][3];
    auto load_a = [&](int s, u32x4 (&f)[3]) {
#pragma unroll
      for (int p = 0; p < 3; ++p) f[p] = ld16(pw + ((int64_t)(c * 16 + s) * 3 + p) * kFrag);
    };
    if (kw < s_end) load_a(kw, fa[0]);
#pragma unroll
    for (int u = 0; u < 16 / KW; ++u) {
      const int s = kw + u * KW;
      if (s < s_end) {
        if (s + KW < s_end) load_a(s + KW, fa[(u + 1) & 1]);
        u32x4 fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[j] = ld16(base + s * 4 * kFrag + rd[j]);
#pragma unroll
        for (int p = 2; p >= 0; --p)  // the smallest part first
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 va[1] = {fa[u & 1][p]}, vb[1] = {fb[j]};
            Op32::step(acc[j], va, vb);
          }
      }
    }
    if (c + 1 < c1) store((c + 1 - c0) & 1);
  }
  if constexpr (KW > 1) {  // add the waves' sums, in the order of kw, through LDS
    float* s = reinterpret_cast<float*>(s_x);
    lds_barrier();
    if (kw > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) s[((wave - WE) * 64 + j * 16 + q) * 64 + lane] = acc[j][q];
    }
    lds_barrier();
    if (kw > 0) return;
#pragma unroll 1  // the loads of all waves' sums at once would not fit the registers
    for (int w = 0; w < KW - 1; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[j][q] += s[((w * WE + we) * 64 + j * 16 + q) * 64 + lane];
  }
  float* out = a.splits > 1 ? a.partial + (int64_t)blockIdx.y * r.E * r.H : r.d_w_router;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int e = eb * kRows + Op32::out_row(lane, q), h = h0 + j * 32 + (lane & 31);
      if (e < r.E && h < r.H) out[(int64_t)e * r.H + h] = acc[j][q];
    }
}

// The splits' sums added in their order, four columns per thread.
__global__ __launch_bounds__(NTH) void route_dw_sum_kernel(const float* __restrict__ partial, int splits, int64_t n,
                                                          float* __restrict__ out) {
  const int64_t at = ((int64_t)blockIdx.x * NTH + threadIdx.x) * 4;
  if (at >= n) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    float p[4];
    unpack(ld16_nt(partial + s * n + at), p);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += p[q];
  }
  st16(out + at, pack(v));
}

// C[m, n] = sum_k A(m, k) B[k, n] in fp32 on v_mfma_f32_32x32x2_f32, B's rows contiguous in n. TRANS: A(m, k) = A[k, m], else
// A[m, k]. 64 x 64 tiles, four waves of 32 x 32, K in steps of 16 through LDS.
template <bool TRANS>
__global__ __launch_bounds__(NTH) void route_grad_gemm_kernel(const float* __restrict__ A, const float* __restrict__ B, int M,
                                                             int N, int K, int lda, float* __restrict__ C) {
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
      s_b[kk][nn] = k0 + kk < K && n0 + nn < N ? B[(int64_t)(k0 + kk) * N + n0 + nn] : 0.f;
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
    if (m < M && n < N) C[(int64_t)m * N + n] = acc[q];
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

namespace {

struct GradSizes {
  int tb, ek, eb, hb, splits, chunks_per_split;
  size_t px, pw, wt, bias, partial, total;
};
GradSizes grad_sizes(int T, int H, int E, int bf16) {
  GradSizes g{};
  g.tb = ceil_div_host(T, kRows);
  g.ek = ceil_div_host(E, kStep);
  g.eb = ceil_div_host(E, kRows);
  g.hb = ceil_div_host(H, kPairCols);
  // d_w_router: parts of the tokens, as many as give every CU a workgroup
  const int chunks = std::max(1, ceil_div_host(T, kDwChunk));
  const int tiles = ceil_div_host(H, kDwCols) * ceil_div_host(g.eb, 8);
  g.chunks_per_split = ceil_div_host(chunks, std::max(1, std::min(chunks, 256 / tiles)));
  g.splits = ceil_div_host(chunks, g.chunks_per_split);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  g.bias = take((size_t)g.tb * E * sizeof(float));
  if (bf16) {
    g.px = take((size_t)g.tb * g.ek * 2 * kFrag);
    g.pw = take((size_t)g.eb * g.tb * 2 * 3 * kFrag);
    g.wt = take((size_t)g.hb * g.ek * 4 * kFrag);
    g.partial = take(g.splits > 1 ? (size_t)g.splits * E * H * sizeof(float) : 0);
  }
  g.total = at;
  return g;
}

template <int WE>
hipError_t launch_dw(const GradArgs& a, hipStream_t stream) {
  const int lds = 2 * kDwChunk * kDwCols * 2, tiles = ceil_div_host(a.r.H, kDwCols);
  const int bias = a.r.d_bias ? ceil_div_host(a.r.E, 64) : 0;
  const hipError_t st = hipFuncSetAttribute(reinterpret_cast<const void*>(route_dw_kernel<WE>),
                                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (st != hipSuccess) return st;
  route_dw_kernel<WE><<<dim3(tiles + bias, a.splits, ceil_div_host(a.eb, 8)), 512, lds, stream>>>(a, tiles);
  return hipGetLastError();
}

template <int WT, int WH>
hipError_t launch_dx(const GradArgs& a, hipStream_t stream) {
  const int lds = WH * a.ek * 4 * kFrag;
  const hipError_t st = hipFuncSetAttribute(reinterpret_cast<const void*>(route_dx_kernel<WT, WH>),
                                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (st != hipSuccess) return st;
  const int cols = ceil_div_host(a.hb, WH), tiles = ceil_div_host(a.tb, 2 * WT);
  route_dx_kernel<WT, WH><<<dim3(cols, std::max(1, std::min(tiles, 256 / cols))), WT * WH * 64, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t route_backward_workspace_bytes(int T, int H, int E, int bf16) { return grad_sizes(T, H, E, bf16).total; }

hipError_t launch_route_backward(const RouteBackward& r, hipStream_t stream) {
  const GradSizes g = grad_sizes(r.T, r.H, r.E, r.bf16);
  unsigned char* ws = static_cast<unsigned char*>(r.workspace);
  GradArgs a{};
  a.r = r;
  a.tb = g.tb;
  a.ek = g.ek;
  a.eb = g.eb;
  a.hb = g.hb;
  a.splits = g.splits;
  a.chunks_per_split = g.chunks_per_split;
  a.bias_part = reinterpret_cast<float*>(ws + g.bias);
  if (r.bf16) {
    a.px = r.d_x ? ws + g.px : nullptr;
    a.pw = r.d_w_router ? ws + g.pw : nullptr;
    a.wt = ws + g.wt;
    a.partial = reinterpret_cast<float*>(ws + g.partial);
  }
  if (r.T > 0) {
    route_grad_prep_kernel<<<a.tb + (a.px ? a.hb * a.eb : 0), NTH, 0, stream>>>(a);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  if (r.bf16) {
    hipError_t st = hipSuccess;
    if (r.d_x && r.T > 0) {
      st = a.ek <= 16 ? launch_dx<4, 2>(a, stream) : launch_dx<8, 1>(a, stream);
      if (st != hipSuccess) return st;
    }
    if (r.d_w_router) {
      st = a.eb <= 1 ? launch_dw<1>(a, stream) : a.eb <= 2 ? launch_dw<2>(a, stream)
           : a.eb <= 4 ? launch_dw<4>(a, stream) : launch_dw<8>(a, stream);
      if (st != hipSuccess) return st;
      if (a.splits > 1) {
        const int64_t n = (int64_t)r.E * r.H;
        route_dw_sum_kernel<<<(unsigned)ceil_div_host64(n / 4, NTH), NTH, 0, stream>>>(a.partial, a.splits, n, r.d_w_router);
      }
    } else if (r.d_bias) {
      route_dbias_kernel<<<ceil_div_host(r.E, 64), 512, 0, stream>>>(a);
    }
    return hipGetLastError();
  }
  if (r.d_x && r.T > 0) {
    const dim3 grid(ceil_div_host(r.H, 64), ceil_div_host(r.T, 64));
    route_grad_gemm_kernel<false><<<grid, NTH, 0, stream>>>(r.d_logits, r.w_router, r.T, r.H, r.E, r.E,
                                                           static_cast<float*>(r.d_x));
  }
  if (r.d_w_router) {
    const dim3 grid(ceil_div_host(r.H, 64), ceil_div_host(r.E, 64));
    route_grad_gemm_kernel<true><<<grid, NTH, 0, stream>>>(r.d_logits, static_cast<const float*>(r.x), r.E, r.H, r.T, r.E,
                                                          r.d_w_router);
  }
  if (r.d_bias) route_dbias_kernel<<<ceil_div_host(r.E, 64), 512, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace moe
