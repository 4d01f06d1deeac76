// Gradients of the combine (moe_combine_backward) and of the router (moe_route_backward).
//
// combine: y[t] = sum_j w[t, j] out[row(t, j)] over kept slots, so d_w[t, j] = dy[t] . out[row] and d_out[row] = w[t, j] dy[t].
//   One workgroup per token reads dy[t] once and its rows once. Bound: HBM (16384 tokens, H 7168, 256 experts of at most 640
//   rows: 344 us, 5.6 TB/s of reads and writes; without d_out 153 us). A row of fewer than 256 slices leaves lanes idle: k 8
//   and H 128 in f32 take 72 us, H 512 in bf16 80, where their bytes are 28 and 55 at a copy's rate; H 2048 in bf16 takes 206,
//   5.5 TB/s.
//
// router: w = softmax over the selected logits, logits = x Wr^T + b. With c_j = w_j (d_w_j - sum_i w_i d_w_i), the gradient of
//   the logits is d_in plus c_j at the selected experts; then d_x = d_logits Wr, d_Wr = d_logits^T x, d_b = the column sums.
#include <algorithm>
#include <type_traits>

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
                                                              const float* __restrict__ topk_w, int T_, int H, int k,
                                                              float* __restrict__ d_w, T* __restrict__ d_out) {
  constexpr int VN = Vec<T>::N;
  __shared__ float s_sum[MOE_MAX_TOPK][NTH / 64];
  const int tid = threadIdx.x;
  const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (t >= T_) return;
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
// The gradient of the logits, T x E values, is small, but a factor of both products (2 T E H operations each).
//   bf16 layers: d_w_router (fp32) is x, exact, times d_logits in three bf16 parts, which hold all of its 24 bits, on bf16 MFMA:
//     every product is exact and the sums are fp32. d_x has two fp32 operands. Each is two fp16 parts, after a power of two for
//     each token and each column of x that puts the largest value at 2^14: off by 2^-22 of itself at most (2^-39 of the largest
//     for what becomes subnormal). Three products, without the one of the two second parts (2^-22 again), so that d_x is what
//     fp32 gives. One fp16 part is not enough, though d_x is rounded to bf16: gradients of a softmax sum to 0 over the
//     experts, what the router's rows share cancels, and 2^-11 of it would stay (rows that are a common one and a hundredth of
//     it their own: d_x off by 0.03 of its norm, with two parts by 0.0017, its rounding). A token or column that holds an
//     infinity or NaN is left out of the product and computed apart in fp32.
//   fp32 layers: fp32 MFMA.
// Fragments: 32 rows x STEP k are the 1 KB that a wave loads at once, lane l row l % 32 and the 16 bytes of k from (l / 32) *
// STEP / 2 on. All operands but x are laid out in fragments by route_grad_prep, their transposes made on the way:
//   route_grad_prep   d_logits, its column sums per 32 tokens, and the fragments of it and of the weight
//   route_dx          the weight's fragments of 32 NJ columns stay in LDS while the tokens stream past
//   route_dw          x is transposed on its way to LDS; the tokens are split over workgroups where the tiles are few
constexpr int kRows = 32, kFrag = 1024;  // rows of a fragment, its bytes
// in place of a power of two: there are infinities among the values; there are NaN
constexpr int kInfinite = 1 << 16, kNan = 1 << 17;

struct GradBf16 {
  using X = bf16_t;
  static constexpr int STEP = 16, PARTS = 3, DXP = 2;  // k of a fragment; parts of d_logits in d_w_router, of d_x's operands
  static constexpr bool SCALED = true;
  static __device__ __forceinline__ void dx(f32x16& acc, u32x4 a, u32x4 b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ void dw(f32x16& acc, u32x4 a, u32x4 b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
  // eight values times 2^e in two fp16 parts; zeros for values that are computed apart
  static __device__ __forceinline__ void dx_operand(const float (&v)[8], int e, u32x4 (&o)[2]) {
    f16x8 hi, lo;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float s = e >= kInfinite ? 0.f : ldexpf(v[q], e);
      hi[q] = (_Float16)s;
      lo[q] = (_Float16)(s - (float)hi[q]);
    }
    o[0] = __builtin_bit_cast(u32x4, hi);
    o[1] = __builtin_bit_cast(u32x4, lo);
  }
  // the values' nearest bf16, and in v what it leaves. What would round to an infinity takes the largest bf16, so that the parts
  // hold every finite value; an infinity or NaN is the part itself and leaves 0.
  static __device__ __forceinline__ u32x4 dw_part(float (&v)[8]) {
    constexpr float kMost = 0x1.fep127f;
    float c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool finite = fabsf(v[q]) < INFINITY;
      c[q] = finite ? fminf(fmaxf(v[q], -kMost), kMost) : v[q];
      v[q] = finite ? v[q] - (float)(bf16_t)c[q] : 0.f;
    }
    return pack(c);
  }
};
struct GradF32 {
  using X = float;
  static constexpr int STEP = 8, PARTS = 1, DXP = 1;
  static constexpr bool SCALED = false;
  static __device__ __forceinline__ void dx(f32x16& acc, u32x4 a, u32x4 b) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[q]), __uint_as_float(b[q]), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ void dw(f32x16& acc, u32x4 a, u32x4 b) { dx(acc, a, b); }
  static __device__ __forceinline__ void dx_operand(const float (&v)[4], int, u32x4 (&o)[1]) { o[0] = pack(v); }
  static __device__ __forceinline__ u32x4 dw_part(float (&v)[4]) { return pack(v); }
};

struct GradArgs {
  RouteBackward r;
  int tb, ek, eb, hb, nj;  // blocks of 32 tokens, k steps and blocks of 32 experts, blocks of 32 nj columns
  unsigned char* px;       // [tb][ek][DXP] fragments: rows tokens, k experts
  unsigned char* pw;       // [eb][tb 32 / STEP][PARTS] fragments: rows experts, k tokens
  unsigned char* wt;       // [hb][ek][DXP][nj] fragments: rows columns of x, k experts; row c of fragment j is column nj c + j
  int* t_exp;              // [32 tb], h_exp [32 nj hb]: the powers of two of the fp16 operands
  int* h_exp;
  float* bias_part;        // [tb][E]
  float* partial;          // [splits][E][H]
  int splits, chunks_per_split;
};

// The power of two that puts a largest value, given by its bits, into [2^14, 2^15); 0 for zero, kInfinite, kNan.
__device__ __forceinline__ int fp16_exp(uint32_t top) {
  if (top >= 0x7f800000u) return top == 0x7f800000u ? kInfinite : kNan;
  if (top == 0) return 0;
  return 15 - (int)(__builtin_amdgcn_frexp_expf(__uint_as_float(top)));
}

// Workgroups [0, tb): 32 tokens each. The others: 32 columns of the weight each.
constexpr int kPrepThreads = 1024;
template <typename G>
__global__ __launch_bounds__(kPrepThreads) void route_grad_prep_kernel(GradArgs a) {
  constexpr int PITCH = MOE_MAX_EXPERTS + 1, WP = kRows + 1, N = G::STEP / 2, NW = kPrepThreads / 64;
  __shared__ float s[kRows * PITCH > MOE_MAX_EXPERTS * WP ? kRows * PITCH : MOE_MAX_EXPERTS * WP];
  __shared__ uint32_t s_top[kPrepThreads / kRows][kRows];
  __shared__ int s_exp[kRows];
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = r.E, k = r.k;
  if ((int)blockIdx.x < a.tb) {
    const int64_t t0 = (int64_t)blockIdx.x * kRows;
    const int n = (int)min((int64_t)kRows, r.T - t0);
    const int ep = a.eb * kRows;  // experts with the padding of a fragment, zeros
    // the selected experts' part: a thread per token, so that an id given twice gets both
    const bool mine = r.d_w && tid < n;
    float w[MOE_MAX_TOPK], d[MOE_MAX_TOPK], sum = 0.f;
    int id[MOE_MAX_TOPK];
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      const int64_t at = (t0 + tid) * k + j;
      const bool in = mine && j < k;
      w[j] = in ? r.w[at] : 0.f;
      d[j] = in ? r.d_w[at] : 0.f;
      id[j] = in ? r.ids[at] : -1;
    }
    for (int i = wave; i < kRows; i += NW)
      for (int e = lane; e < ep; e += 64) s[i * PITCH + e] = r.d_in && i < n && e < E ? r.d_in[(t0 + i) * E + e] : 0.f;
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOPK; ++j)
        if (j < k) sum = fmaf(w[j], d[j], sum);
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOPK; ++j)
        if (id[j] >= 0 && id[j] < E) s[tid * PITCH + id[j]] += w[j] * (d[j] - sum);
    }
    __syncthreads();
    for (int i = wave; i < kRows; i += NW) {
      uint32_t top = 0;
      for (int e = lane; e < E; e += 64) {
        const float v = s[i * PITCH + e];
        if (i < n) r.d_logits[(t0 + i) * E + e] = v;
        top = max(top, __float_as_uint(v) & 0x7fffffffu);
      }
      if (G::SCALED && a.px) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
        if (lane == 0) {
          s_exp[i] = fp16_exp(top);
          a.t_exp[t0 + i] = s_exp[i];
        }
      }
    }
    if (r.d_bias)
      for (int e = tid; e < E; e += kPrepThreads) {
        float v = 0.f;
        for (int i = 0; i < n; ++i) v += s[i * PITCH + e];
        a.bias_part[(int64_t)blockIdx.x * E + e] = v;
      }
    if (a.pw)
      for (int i = tid; i < a.eb * (kRows / G::STEP) * 64; i += kPrepThreads) {
        const int l = i & 63, step = (i >> 6) % (kRows / G::STEP), b = (i >> 6) / (kRows / G::STEP);
        float v[N];
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = s[(step * G::STEP + (l >> 5) * N + q) * PITCH + b * kRows + (l & 31)];
        unsigned char* f = a.pw + (((int64_t)b * a.tb + blockIdx.x) * (kRows / G::STEP) + step) * G::PARTS * kFrag + l * 16;
#pragma unroll
        for (int p = 0; p < G::PARTS; ++p) st16(f + p * kFrag, G::dw_part(v));
      }
    __syncthreads();  // s_exp
    if (a.px)
      for (int i = tid; i < a.ek * 64; i += kPrepThreads) {
        const int l = i & 63, step = i >> 6;
        float v[N];
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = s[(l & 31) * PITCH + step * G::STEP + (l >> 5) * N + q];
        u32x4 o[G::DXP];
        G::dx_operand(v, G::SCALED ? s_exp[l & 31] : 0, o);
#pragma unroll
        for (int p = 0; p < G::DXP; ++p)
          st16(a.px + (((int64_t)blockIdx.x * a.ek + step) * G::DXP + p) * kFrag + l * 16, o[p]);
      }
    return;
  }
  const int c = tid & 31, g = tid >> 5;  // column of the 32, and which experts
  const int h0 = (blockIdx.x - a.tb) * kRows, ep = a.ek * G::STEP;
  uint32_t top = 0;
  for (int e = g; e < ep; e += kPrepThreads / kRows) {
    const float v = e < E && h0 + c < r.H ? r.w_router[(int64_t)e * r.H + h0 + c] : 0.f;
    s[e * WP + c] = v;
    top = max(top, __float_as_uint(v) & 0x7fffffffu);
  }
  if constexpr (G::SCALED) {
    s_top[g][c] = top;
    __syncthreads();
    if (tid < kRows) {
      for (int i = 1; i < kPrepThreads / kRows; ++i) top = max(top, s_top[i][c]);
      s_exp[c] = fp16_exp(top);
      a.h_exp[h0 + c] = s_exp[c];
    }
  }
  __syncthreads();
  const int per = 32 / a.nj;  // this workgroup's rows of each fragment: column nj row + j
  for (int i = tid; i < a.ek * a.nj * 2 * per; i += kPrepThreads) {
    const int row = i % per, half = i / per & 1, j = i / (2 * per) % a.nj, step = i / (2 * per * a.nj);
    const int col = a.nj * row + j, b = h0 / (32 * a.nj), row0 = h0 % (32 * a.nj) / a.nj;
    float v[N];
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = s[(step * G::STEP + half * N + q) * WP + col];
    u32x4 o[G::DXP];
    G::dx_operand(v, G::SCALED ? s_exp[col] : 0, o);
#pragma unroll
    for (int p = 0; p < G::DXP; ++p)
      st16(a.wt + ((((int64_t)b * a.ek + step) * G::DXP + p) * a.nj + j) * kFrag + (half * 32 + row0 + row) * 16, o[p]);
  }
}

// d_x of a block's tokens and a lane's NJ columns where either holds a NaN, which all of its products are, or an infinity: fp32
// products, eight at once on their way, until they are NaN. 4096 tokens, H 7168, 256 experts, the call: 123 us without, 192 where
// every value is NaN, 178 with one infinity, 8.1 ms with one in every token.
template <int NJ>
__device__ __forceinline__ void route_dx_apart(const GradArgs& a, int64_t t0, int h, int lane) {
  const RouteBackward& r = a.r;
#pragma unroll 1
  for (int i = 0; i < 16 * NJ; ++i) {
    const int64_t t = t0 + Op32::out_row(lane, i / NJ);
    const int c = h + i % NJ;
    if (t >= r.T || c >= r.H) continue;
    const int most = max(a.t_exp[t], a.h_exp[c]);
    if (most < kInfinite) continue;
    float v = most == kNan ? __uint_as_float(0x7fc00000u) : 0.f;
#pragma unroll 1
    for (int e0 = 0; e0 < r.E && v == v; e0 += 8) {
      float d[8], w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const bool in = e0 + q < r.E;
        d[q] = in ? r.d_logits[t * r.E + e0 + q] : 0.f;
        w[q] = in ? r.w_router[(int64_t)(e0 + q) * r.H + c] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) v = fmaf(d[q], w[q], v);
    }
    static_cast<bf16_t*>(r.d_x)[t * r.H + c] = (bf16_t)v;
  }
}

// d_x: a wave computes 32 TI tokens x 32 NJ columns, eight waves. The columns' fragments are in LDS for good; the tokens' come from
// memory D - 1 steps ahead, across the ends of the token tiles. A lane has NJ neighbouring columns of a row.
constexpr int kDxWaves = 8;
template <typename G>
int dx_lds(int ek, int nj) {  // the fragments and, behind them, the columns' powers of two
  return ek * G::DXP * nj * kFrag + (G::SCALED ? 32 * nj * (int)sizeof(int) : 0);
}
template <typename G, int NJ, int TI, int D>
__device__ __forceinline__ void route_dx(const GradArgs& a, unsigned char* s_w, int block_x, int block_y, int grid_y) {
  constexpr int WT = kDxWaves, NT = WT * 64, P = G::DXP;
  using X = typename G::X;
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wt = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int block = a.ek * P * NJ * kFrag;
  for (int i = tid * 16; i < block; i += NT * 16 * 8) {
    u32x4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q * NT * 16 < block) v[q] = ld16(a.wt + (int64_t)block_x * block + i + q * NT * 16);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q * NT * 16 < block) st16(s_w + i + q * NT * 16, v[q]);
  }
  const int tiles = (a.tb - wt * TI + TI * WT - 1) / (TI * WT);  // of 32 TI WT tokens, those where this wave has any
  u32x4 fa[D][TI][P];  // 32-token blocks
  int tile = block_y, step = 0, ltile = block_y, lstep = 0;
  // the next step that is not on its way yet; past the last one a valid address, as a branch around loads makes the compiler
  // wait for all of them
  auto load = [&](u32x4 (&f)[TI][P]) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int tb = min((ltile * WT + wt) * TI + i, a.tb - 1);
#pragma unroll
      for (int p = 0; p < P; ++p) f[i][p] = ld16(a.px + (((int64_t)tb * a.ek + lstep) * P + p) * kFrag + lane * 16);
    }
    if (++lstep == a.ek) {
      lstep = 0;
      ltile += grid_y;
    }
  };
  f32x16 acc[TI][NJ];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  };
  clear();
#pragma unroll
  for (int i = 0; i < D - 1; ++i) load(fa[i]);
  if (G::SCALED && tid < 32 * NJ) reinterpret_cast<int*>(s_w + block)[tid] = a.h_exp[block_x * 32 * NJ + tid];
  __syncthreads();
  auto one = [&](auto U) {
    constexpr int u = decltype(U)::value;
    load(fa[(u + D - 1) % D]);
    u32x4 fb[P][NJ];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < NJ; ++j) fb[p][j] = ld16(s_w + ((step * P + p) * NJ + j) * kFrag + lane * 16);
#pragma unroll
    for (int p = 2 * P - 2; p >= 0; --p)  // the parts' products, the smaller ones first: (0, 1), (1, 0), (0, 0)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) G::dx(acc[i][j], fa[u][i][p & 1], fb[p >> 1][j]);
    if (++step == a.ek) {
      const int h = block_x * 32 * NJ + NJ * (lane & 31);
      const int* s_he = reinterpret_cast<const int*>(s_w + block) + NJ * (lane & 31);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int tb = (tile * WT + wt) * TI + i;
        const int64_t t0 = (int64_t)tb * kRows;
        // the powers of two of the block's tokens, by scalar loads: vector loads would wait for the fragments on their way
        const auto* te = (const __attribute__((address_space(4))) int*)(a.t_exp + (int64_t)min(tb, a.tb - 1) * kRows);
        int he[NJ];
        int most = 0;  // the largest of the powers, or 0: kInfinite or kNan where something has to be computed apart
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          he[j] = G::SCALED ? s_he[j] : 0;
          most = max(most, he[j]);
        }
        if (t0 < r.T) {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int64_t t = t0 + Op32::out_row(lane, q);
            const int ti = !G::SCALED ? 0 : lane < 32 ? te[Op32::out_row(0, q)] : te[Op32::out_row(32, q)];
            most = max(most, ti);
            if (t < r.T && h < r.H) {
              X* o = static_cast<X*>(r.d_x) + t * r.H + h;
              float v[NJ];
#pragma unroll
              for (int j = 0; j < NJ; ++j) v[j] = G::SCALED ? ldexpf(acc[i][j][q], -ti - he[j]) : acc[i][j][q];
              if constexpr (sizeof(X) == 4 && NJ == 4) *reinterpret_cast<u32x4*>(o) = pack(v);
              else if constexpr (sizeof(X) == 4) *reinterpret_cast<f32x2*>(o) = f32x2{v[0], v[1]};
              else if constexpr (NJ == 2) __builtin_nontemporal_store(pack2_bf16(v[0], v[1]), reinterpret_cast<uint32_t*>(o));
              else  // (non-temporal: 29.4 -> 27.7 us with operands of one part)
                __builtin_nontemporal_store(u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])},
                                            reinterpret_cast<u32x2*>(o));
            }
          }
          if constexpr (G::SCALED)
            if (most >= kInfinite) route_dx_apart<NJ>(a, t0, h, lane);
        }
      }
      clear();
      step = 0;
      tile += grid_y;
    }
  };
  while (tile < tiles) {
    one(std::integral_constant<int, 0>{});
    if (tile < tiles) one(std::integral_constant<int, 1>{});
    if constexpr (D == 4) {
      if (tile < tiles) one(std::integral_constant<int, 2>{});
      if (tile < tiles) one(std::integral_constant<int, 3>{});
    }
  }
}
// PER_CU workgroups share a CU
template <typename G, int NJ, int TI, int D, int PER_CU>
__global__ __launch_bounds__(kDxWaves * 64, 2 * PER_CU) void route_dx_kernel(GradArgs a) {
  static_assert(D == 2 || D == 4, "the loop over the steps");
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  route_dx<G, NJ, TI, D>(a, smem, blockIdx.x, blockIdx.y, gridDim.y);
}

// Column sums of d_logits from those of 32 tokens: 64 columns per workgroup of NW waves, their sums added in order.
template <int NW>
__device__ __forceinline__ void bias_sums(const GradArgs& a, int block, double* s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = block * 64 + lane;
  double v = 0.0;
  if (e < a.r.E)
    for (int i0 = wave; i0 < a.tb; i0 += 8 * NW) {  // eight loads in flight
      float p[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) p[q] = i0 + q * NW < a.tb ? a.bias_part[(int64_t)(i0 + q * NW) * a.r.E + e] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += (double)p[q];
    }
  s[wave * 64 + lane] = v;
  __syncthreads();
  if (wave == 0 && e < a.r.E) {
    v = 0.0;
    for (int i = 0; i < NW; ++i) v += s[i * 64 + lane];
    a.r.d_bias[e] = (float)v;
  }
}
__global__ __launch_bounds__(512) void route_dbias_kernel(GradArgs a) {
  __shared__ double s[512];
  bias_sums<8>(a, blockIdx.x, s);
}

// d_w_router: eight waves, WE along the experts (32 each) and 8 / WE along the tokens, whose sums are added in the end; 128
// columns of x. Tokens go in chunks of 16 steps: a thread loads 8 tokens x 16 bytes of the next chunk while this one is
// multiplied. In LDS the chunk is fragments [step][4 column blocks]; in a fragment the 16 bytes of column c are at place
// c ^ (its group of 8 in the 128 columns), so that the writes of a wave, at a stride of 4 or 8 columns, touch all banks.
// Workgroups past the column tiles add up the bias. A second chunk of x on its way changed nothing (16000 tokens, H 4096, 8
// experts: 43 us, 3.1 TB/s); two workgroups of four waves per CU were slower (52). 4096 tokens, H 7168, 256 experts: 50 us, the
// matrix units busy 55 % of it.
constexpr int kDwCols = 128;
constexpr int kDwSteps = 16, kDwChunkBytes = kDwSteps * 4 * kFrag;
template <typename G, int WE>
__device__ __forceinline__ void route_dw(const GradArgs& a, unsigned char* s_x, int block, int col_tiles) {
  constexpr int NW = 8, KW = NW / WE, P = G::PARTS, VN = Vec<typename G::X>::N, CT = kDwSteps * G::STEP;
  static_assert(CT / 8 * (kDwCols / VN) == NW * 64, "a thread loads 8 tokens x 16 bytes of a chunk");
  const RouteBackward& r = a.r;
  const int tid = threadIdx.x, lane = tid & 63;
  // a workgroup's unit: splits of the tokens are the slowest index and an XCD takes neighbouring units, so that its L2 holds the
  // d_logits of one split
  const int e_tiles = (a.eb + 7) / 8, units = col_tiles * e_tiles * a.splits, per = (units + 7) >> 3;
  const int unit = (block & 7) * per + (block >> 3);
  if (block >= per * 8) {
    bias_sums<NW>(a, block - per * 8, reinterpret_cast<double*>(s_x));
    return;
  }
  if (unit >= units) return;
  const int split = unit / (col_tiles * e_tiles), e_tile = unit / col_tiles % e_tiles;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int we = wave % WE, kw = wave / WE;
  const int eb = e_tile * 8 + we;  // this wave's 32 experts
  const int h0 = unit % col_tiles * kDwCols;
  const int steps = a.tb * (kRows / G::STEP), chunks = (steps + kDwSteps - 1) / kDwSteps;
  const int c0 = split * a.chunks_per_split, c1 = min(chunks, c0 + a.chunks_per_split);
  const typename G::X* x = static_cast<const typename G::X*>(r.x);
  const int gv = tid % (kDwCols / VN), t8 = tid / (kDwCols / VN);  // this thread's VN columns and 8 tokens of a chunk
  const bool in_h = h0 + gv * VN < r.H;
  u32x4 raw[8];
  // rows of chunk c; past the last token, and in lanes past H, the offset reads zeros. All loads here are unconditional: a
  // branch around some makes the compiler wait for more of them than it needs.
  const int voff = in_h ? (t8 * 8 * r.H + h0 + gv * VN) * (int)sizeof(*x) : 0x7ffffff0;
  auto load = [&](int c) {
    const int64_t t0 = min((int64_t)c * CT, (int64_t)r.T);
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(x + t0 * r.H), (short)0, (int)(min((int64_t)CT, r.T - t0) * r.H * (int)sizeof(*x)), 0x00020000);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      raw[i] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, in_h ? voff + i * r.H * (int)sizeof(*x) : voff, 0, 2));
  };
  auto store = [&](int slot) {
    const int col = gv * VN, g8 = col >> 3;
    unsigned char* base = s_x + slot * kDwChunkBytes + (((t8 * 8 / G::STEP) * 4 + (col >> 5)) * 64 + (col & 24)) * 16;
#pragma unroll
    for (int c = 0; c < VN; ++c) {
      unsigned char* o = base + ((((col & 7) + c) ^ g8) & 7) * 16;
      if constexpr (VN == 8) {
        u32x4 v;
#pragma unroll
        for (int p = 0; p < 4; ++p)  // tokens 2 p and 2 p + 1 of column c
          v[p] = __builtin_amdgcn_perm(raw[2 * p + 1][c >> 1], raw[2 * p][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
        st16(o + (t8 & 1) * 512, v);
      } else {
        st16(o, u32x4{raw[0][c], raw[1][c], raw[2][c], raw[3][c]});
        st16(o + 512, u32x4{raw[4][c], raw[5][c], raw[6][c], raw[7][c]});
      }
    }
  };
  f32x16 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[j][q] = 0.f;
  const unsigned char* pw = a.pw + (int64_t)min(eb, a.eb - 1) * steps * P * kFrag + lane * 16;
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
  constexpr int U = kDwSteps / KW, D = U < 4 ? U : 4;  // a wave's steps of a chunk; buffers of d_logits' fragments
  static_assert(U % D == 0, "a chunk takes every buffer as often");
  u32x4 fa[D][P];
  auto load_a = [&](int s, u32x4 (&f)[P]) {  // step s of all
#pragma unroll
    for (int p = 0; p < P; ++p) f[p] = ld16(pw + ((int64_t)max(0, min(s, steps - 1)) * P + p) * kFrag);
  };
  if (steps > 0) {
#pragma unroll
    for (int u = 0; u < D - 1; ++u) load_a(c0 * kDwSteps + kw + u * KW, fa[u]);
  }
  // One chunk; its last steps are past the tokens in the last chunk only. The columns' fragments are read one step ahead.
  auto chunk = [&](int c) {
    const unsigned char* base = s_x + ((c - c0) & 1) * kDwChunkBytes;
    u32x4 fb[2][4];
    auto read_b = [&](int s, u32x4 (&f)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = ld16(base + s * 4 * kFrag + rd[j]);
    };
    read_b(kw, fb[0]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = kw + u * KW;
      load_a(c * kDwSteps + s + (D - 1) * KW, fa[(u + D - 1) % D]);
      if (u == 0) load(c + 1);  // (spread over the steps: 65 against 56 us)
      if (u + 1 < U) read_b(s + KW, fb[(u + 1) & 1]);
      if (c * kDwSteps + s < steps) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p)  // the smallest part first
#pragma unroll
          for (int j = 0; j < 4; ++j) G::dw(acc[j], fa[u % D][p], fb[u & 1][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int c = c0; c < c1; ++c) {
    lds_barrier();  // chunk c is in LDS, and chunk c - 1 has been read
    chunk(c);
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
  float* out = a.splits > 1 ? a.partial + (int64_t)split * r.E * r.H : r.d_w_router;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int e = eb * kRows + Op32::out_row(lane, q), h = h0 + j * 32 + (lane & 31);
      if (e < r.E && h < r.H) out[(int64_t)e * r.H + h] = acc[j][q];
    }
}
template <typename G, int WE>
__global__ __launch_bounds__(512) void route_dw_kernel(GradArgs a, int col_tiles) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  route_dw<G, WE>(a, smem, blockIdx.x, col_tiles);
}

// Both in one launch, where their workgroups fit the CUs side by side: dx's hb x dx_y, then dw's.
template <typename G, int NJ, int WE>
__global__ __launch_bounds__(512) void route_dx_dw_kernel(GradArgs a, int dx_y, int col_tiles) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int b = blockIdx.x, n = a.hb * dx_y;
  if (b < n) route_dx<G, NJ, 1, 4>(a, smem, b % a.hb, b / a.hb, dx_y);
  else route_dw<G, WE>(a, smem, b - n, col_tiles);
}

// The splits' sums added in their order, four columns per thread.
__global__ __launch_bounds__(NTH) void route_dw_sum_kernel(const float* __restrict__ partial, int splits, int64_t n,
                                                          float* __restrict__ out) {
  const int64_t at = ((int64_t)blockIdx.x * NTH + threadIdx.x) * 4;
  if (at >= n) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 8) {  // eight loads in flight
    u32x4 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = s0 + i < splits ? ld16_nt(partial + (s0 + i) * n + at) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float p[4];
      unpack(raw[i], p);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += p[q];
    }
  }
  st16(out + at, pack(v));
}

}  // namespace

hipError_t launch_combine_backward(const void* dy, int bf16, const void* out_buf, const moe_layout_t& L,
                                   const float* topk_w, float* d_w, void* d_out, hipStream_t stream) {
  const int nvec = L.H / (bf16 ? 8 : 4);
#define MOE_GO(TY, VPT)                                                                                            \
  combine_backward_kernel<TY, VPT>                                                                                 \
      <<<token_grid(L.T), NTH, 0, stream>>>(static_cast<const TY*>(dy), static_cast<const TY*>(out_buf), L.pair_row, topk_w, \
                                            L.T, L.H, L.k, d_w, static_cast<TY*>(d_out))
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
  int tb, ek, eb, hb, nj, splits, chunks_per_split;
  size_t px, pw, wt, t_exp, h_exp, bias, partial, total;
};
template <typename G>
GradSizes grad_sizes(int T, int H, int E) {
  GradSizes g{};
  g.tb = ceil_div_host(T, kRows);
  g.ek = ceil_div_host(E, G::STEP);
  g.eb = ceil_div_host(E, kRows);
  // the weight's fragments of 32 nj columns take DXP KB ek nj of LDS, 128 KB at most
  g.nj = g.ek * G::DXP <= 32 ? 4 : 2;
  g.hb = ceil_div_host(H, 32 * g.nj);
  // d_w_router: parts of the tokens, as many as give every CU a workgroup
  const int chunks = std::max(1, ceil_div_host(T, kDwSteps * G::STEP));
  const int tiles = ceil_div_host(H, kDwCols) * ceil_div_host(g.eb, 8);
  // (a chunk of few experts' steps takes less than the launch that adds the parts)
  g.chunks_per_split = std::max(g.eb <= 2 ? 3 : 1, ceil_div_host(chunks, std::max(1, std::min(chunks, 256 / tiles))));
  g.splits = ceil_div_host(chunks, g.chunks_per_split);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  g.bias = take((size_t)g.tb * E * sizeof(float));
  g.px = take((size_t)g.tb * g.ek * G::DXP * kFrag);
  g.pw = take((size_t)g.eb * g.tb * (kRows / G::STEP) * G::PARTS * kFrag);
  g.wt = take((size_t)g.hb * g.ek * G::DXP * g.nj * kFrag);
  g.t_exp = take((size_t)g.tb * kRows * sizeof(int));
  g.h_exp = take((size_t)g.hb * 32 * g.nj * sizeof(int));
  g.partial = take(g.splits > 1 ? (size_t)g.splits * E * H * sizeof(float) : 0);
  g.total = at;
  return g;
}

template <typename G, int WE>
hipError_t launch_dw(const GradArgs& a, hipStream_t stream) {
  const int lds = 2 * kDwChunkBytes, tiles = ceil_div_host(a.r.H, kDwCols);
  const int bias = a.r.d_bias ? ceil_div_host(a.r.E, 64) : 0;
  const int units = tiles * a.splits * ceil_div_host(a.eb, 8);
  route_dw_kernel<G, WE><<<ceil_div_host(units, 8) * 8 + bias, 512, lds, stream>>>(a, tiles);
  return hipGetLastError();
}

// Both products in one launch, if they fit the CUs together (17 tokens, H 1216, 215 experts: 23 -> 15 us with the preparation
// when d_x's operands had one part; 17 with two); returns whether they did
template <typename G, int NJ, int WE>
bool launch_dx_dw(const GradArgs& a, hipStream_t stream) {
  const int tiles = ceil_div_host(a.r.H, kDwCols), units = tiles * a.splits * ceil_div_host(a.eb, 8);
  const int dx_y = ceil_div_host(a.tb, 8), bias = a.r.d_bias ? ceil_div_host(a.r.E, 64) : 0;
  if ((int64_t)a.hb * dx_y + units > 256) return false;
  const int lds = std::max(2 * kDwChunkBytes, dx_lds<G>(a.ek, NJ));
  route_dx_dw_kernel<G, NJ, WE>
      <<<a.hb * dx_y + ceil_div_host(units, 8) * 8 + bias, 512, lds, stream>>>(a, dx_y, tiles);
  return true;
}

template <typename G, int NJ, int TI, int D, int PER_CU>
hipError_t launch_dx(const GradArgs& a, hipStream_t stream) {
  const int tiles = ceil_div_host(a.tb, TI * kDxWaves);
  const dim3 grid(a.hb, std::max(1, std::min(tiles, PER_CU * 256 / a.hb)));
  route_dx_kernel<G, NJ, TI, D, PER_CU><<<grid, kDxWaves * 64, dx_lds<G>(a.ek, NJ), stream>>>(a);
  return hipGetLastError();
}

template <typename G>
hipError_t launch_route_backward_t(const RouteBackward& r, hipStream_t stream) {
  const GradSizes g = grad_sizes<G>(r.T, r.H, r.E);
  unsigned char* ws = static_cast<unsigned char*>(r.workspace);
  GradArgs a{};
  a.r = r;
  a.tb = g.tb;
  a.ek = g.ek;
  a.eb = g.eb;
  a.hb = g.hb;
  a.nj = g.nj;
  a.splits = g.splits;
  a.chunks_per_split = g.chunks_per_split;
  a.bias_part = reinterpret_cast<float*>(ws + g.bias);
  a.px = r.d_x ? ws + g.px : nullptr;
  a.pw = r.d_w_router ? ws + g.pw : nullptr;
  a.wt = ws + g.wt;
  a.t_exp = reinterpret_cast<int*>(ws + g.t_exp);
  a.h_exp = reinterpret_cast<int*>(ws + g.h_exp);
  a.partial = reinterpret_cast<float*>(ws + g.partial);
  hipError_t st = hipSuccess;
  bool joint = false;
  if (r.T > 0) {
    route_grad_prep_kernel<G><<<a.tb + (r.d_x ? a.hb * a.nj : 0), kPrepThreads, 0, stream>>>(a);
    st = hipGetLastError();
    if (st == hipSuccess && r.d_x && r.d_w_router) {
      if (a.nj == 4)
        joint = a.eb <= 1 ? launch_dx_dw<G, 4, 1>(a, stream) : a.eb <= 2 ? launch_dx_dw<G, 4, 2>(a, stream)
                : a.eb <= 4 ? launch_dx_dw<G, 4, 4>(a, stream) : launch_dx_dw<G, 4, 8>(a, stream);
      else joint = launch_dx_dw<G, 2, 8>(a, stream);
    }
    if (st == hipSuccess && r.d_x && !joint) {
      if constexpr (G::SCALED) {
        // Two workgroups per CU, whose stores and products overlap, where half the LDS and half the registers do (16 experts,
        // 16384 tokens, H 4096: 29.5 us against 38.5 with one; 64 experts, 4096 tokens, H 7168: 23.2 against 26.9). With one,
        // 64 tokens per wave take every fragment of the weight out of LDS half as often, which pays with two blocks of
        // columns, given tokens for all waves (4096 tokens, H 7168, 384 and 512 experts: 82 and 105 us against 89 and 117;
        // 240 tokens, H 20480, 512 experts: 40 against 33; four blocks, 256 experts: 53 either way).
        if (a.nj == 2) st = a.tb > kDxWaves ? launch_dx<G, 2, 2, 4, 1>(a, stream) : launch_dx<G, 2, 1, 4, 1>(a, stream);
        else st = a.ek <= 8 ? launch_dx<G, 4, 1, 2, 2>(a, stream) : launch_dx<G, 4, 1, 4, 1>(a, stream);
      } else {
        // (256 experts, 4096 tokens, H 7168: 149 us, 101 TFLOP/s; 64 tokens per wave took as long)
        st = a.nj == 2 ? launch_dx<G, 2, 1, 4, 2>(a, stream) : launch_dx<G, 4, 1, 4, 2>(a, stream);
      }
    }
    if (st != hipSuccess) return st;
  }
  if (r.d_w_router) {
    if (!joint)
      st = a.eb <= 1 ? launch_dw<G, 1>(a, stream) : a.eb <= 2 ? launch_dw<G, 2>(a, stream)
           : a.eb <= 4 ? launch_dw<G, 4>(a, stream) : launch_dw<G, 8>(a, stream);
    else st = hipGetLastError();
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

}  // namespace

size_t route_backward_workspace_bytes(int T, int H, int E, int bf16) {
  return bf16 ? grad_sizes<GradBf16>(T, H, E).total : grad_sizes<GradF32>(T, H, E).total;
}

hipError_t launch_route_backward(const RouteBackward& r, hipStream_t stream) {
  return r.bf16 ? launch_route_backward_t<GradBf16>(r, stream) : launch_route_backward_t<GradF32>(r, stream);
}

}  // namespace moe
