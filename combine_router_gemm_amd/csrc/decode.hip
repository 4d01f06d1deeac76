// The whole MoE layer for a few tokens (T <= 32): moe_layer_decode and moe_layer_decode_w4.
//
//   logits = x Wr^T + b            decode_route_kernel
//   top-k, softmax, capacity       choose(), by every workgroup of the next kernels for itself
//   h = silu(x Wg^T) * (x Wu^T)    decode_gate_up_kernel, per chosen expert
//   y = sum_j w_j h_j Wd^T         decode_down_kernel
//
// What bounds it: the bytes of the chosen experts' weights, each read once. The weights are the M operand of the
// matrix unit (16 output columns per tile) and the tokens its N operand (NB blocks of 16): token t is always column
// t, so an expert's products of tokens that did not choose it are computed along (the matrix unit has the time) and
// dropped by a select, never by a multiplication with zero. No row is gathered or scattered and no partial
// result is added atomically: the down kernel adds a token's experts in expert order in registers.
#include <algorithm>
#include <climits>
#include <type_traits>
#include <climits>

#include "common.h"
#include "kernels.h"
#include "mfma.h"
#include "topk.h"
#include "w4.h"

namespace moe {

namespace {

constexpr int DEC_NW = 8;                // waves per workgroup: they split K
constexpr int DEC_NTH = DEC_NW * 64;
constexpr int DEC_PAIRS = MOE_DECODE_MAX_TOKENS * MOE_MAX_TOPK;
static_assert(DEC_NTH >= MOE_MAX_EXPERTS, "choose() has a thread per expert");

struct DecodeArgs {
  const void* x;        // [T, H]
  const float* logits;  // [T, E]
  int T, H, E, El, k, C, F;
  const void* w_gu;     // [El, 2F, H], or its packed codes
  const void* w_dn;     // [El, H, F]
  const uint8_t* s_gu;  // scales of packed weights
  const uint8_t* s_dn;
  int* ids;             // [T, k]
  float* wts;           // [T, k]
  void* y;              // [T, H]
  void* h;              // [T * k, F]: fp32, or for bf16 layers the bf16 nearest to h and then [T * k, F] its remainder
};

// ------------------------------------------------------------------------------------------------
// router
// ------------------------------------------------------------------------------------------------
// One workgroup per expert and TB tokens: its 256 threads share the fp32 weight row, every thread takes eight
// consecutive k at a time (exact products, at most ceil(H / 2048) * 8 fp32 additions in a row), then a fixed
// tree of additions.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float (&v)[8]) {
  unpack(ld16(p), v);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  unpack(ld16(p), *reinterpret_cast<float(*)[4]>(&v[0]));
  unpack(ld16(p + 4), *reinterpret_cast<float(*)[4]>(&v[4]));
}

template <typename T, int TB>
__global__ __launch_bounds__(256) void decode_route_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                                           const float* __restrict__ bias, int64_t bias_stride, int T_,
                                                           int H, int E, float* __restrict__ logits) {
  __shared__ float s_sum[4][TB];
  const int e = blockIdx.x, t0 = blockIdx.y * TB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float acc[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) acc[j] = 0.f;
  for (int c = tid * 8; c < H; c += 2048) {
    float wv[8];
    load8(w + (int64_t)e * H + c, wv);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      float xv[8];
      load8(x + (int64_t)min(t0 + j, T_ - 1) * H + c, xv);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[j] = fmaf(xv[q], wv[q], acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const float s = wave_sum(acc[j]);
    if (lane == 0) s_sum[wave][j] = s;
  }
  __syncthreads();
  if (tid < TB && t0 + tid < T_) {
    float v = (s_sum[0][tid] + s_sum[1][tid]) + (s_sum[2][tid] + s_sum[3][tid]);
    if (bias) v += bias[(int64_t)(t0 + tid) * bias_stride + e];
    logits[(int64_t)(t0 + tid) * E + e] = v;
  }
}

// ------------------------------------------------------------------------------------------------
// choice of experts
// ------------------------------------------------------------------------------------------------
struct Choice {
  int n;                      // experts with a kept pair, ascending
  int wcnt[DEC_NW];
  int expert[DEC_PAIRS];
  uint32_t mask[DEC_PAIRS];   // bit t: token t is kept there
  uint8_t slot[DEC_PAIRS][MOE_DECODE_MAX_TOKENS];  // its slot
  int ids[DEC_PAIRS];
  float w[DEC_PAIRS];
  uint32_t chosen[MOE_MAX_EXPERTS];
  uint16_t place[MOE_MAX_EXPERTS];
};

// Top-k, softmax and capacity of every token from the logits, by a whole workgroup: a wave per token, expert
// lane * V + i in the lane's i-th value; each of the k rounds takes the wave's largest key, the lowest expert among
// equals (moe_route's rule: -0 == +0, a NaN ranks as -inf). Repeated by every workgroup: it takes about as long as
// one more dependent launch would, and nothing has to be passed on.
__device__ __forceinline__ void choose(const DecodeArgs& a, Choice& c, bool write) {
  constexpr int VMAX = MOE_MAX_EXPERTS / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = (a.E + 63) / 64;
  c.chosen[tid] = 0;
  __syncthreads();
  for (int t = wave; t < a.T; t += DEC_NW) {
    int key[VMAX];
#pragma unroll
    for (int i = 0; i < VMAX; ++i) {
      const int e = lane * V + i;
      key[i] = INT_MIN;
      if (i < V && e < a.E) {
        const float s = a.logits[(int64_t)t * a.E + e] + 0.0f;  // -0 -> +0
        key[i] = float_key(s == s ? s : -INFINITY);
      }
    }
    float sel_v[MOE_MAX_TOPK];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j) {
      sel_v[j] = 0.f;
      if (j < a.k) {
        int head = INT_MIN, at = 0;
#pragma unroll
        for (int i = 0; i < VMAX; ++i)
          if (key[i] > head) {
            head = key[i];
            at = i;
          }
        const int m = wave_max_i32(head);
        const int wl = __builtin_ctzll(__ballot(head == m));  // k <= E: m is a present value's key
        const int e = __builtin_amdgcn_readlane(lane * V + at, wl);
        sel_v[j] = key_float(m);
        if (lane == j) mine = e;
#pragma unroll
        for (int i = 0; i < VMAX; ++i)
          if (lane == wl && i == at) key[i] = INT_MIN;
      }
    }
    float sum = 0.f, z_mine = 0.f;
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOPK; ++j)
      if (j < a.k) {
        const float z = expf(sel_v[j] - sel_v[0]);
        sum += z;
        if (j == lane) z_mine = z;
      }
    if (lane < a.k) {
      c.ids[t * a.k + lane] = mine;
      c.w[t * a.k + lane] = z_mine / sum;
      atomicOr(&c.chosen[mine], 1u << t);
      if (write) {
        a.ids[t * a.k + lane] = mine;
        a.wts[t * a.k + lane] = z_mine / sum;
      }
    }
  }
  __syncthreads();
  // the first C tokens of every expert; experts with any, in ascending order
  uint32_t m = tid < a.E ? c.chosen[tid] : 0u;
  for (int over = __popc(m) - a.C; over > 0; --over) m &= ~(0x80000000u >> __clz(m));
  const uint64_t b = __ballot(m != 0);
  if (lane == 0) c.wcnt[wave] = __popcll(b);
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < DEC_NW; ++w) base += w < wave ? c.wcnt[w] : 0;
  if (tid < a.E) c.chosen[tid] = m;
  if (m != 0) {
    const int i = base + __popcll(b & lanemask_lt());
    c.expert[i] = tid;
    c.mask[i] = m;
    c.place[tid] = (uint16_t)i;
  }
  if (tid == DEC_NTH - 1) c.n = base + __popcll(b);
  __syncthreads();
  for (int p = tid; p < a.T * a.k; p += DEC_NTH) {
    const int e = c.ids[p], t = p / a.k;
    if ((c.chosen[e] >> t) & 1u) c.slot[c.place[e]][t] = (uint8_t)(p - t * a.k);
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------------------------
// operands
// ------------------------------------------------------------------------------------------------
template <typename T>
struct DecOp;
template <>
struct DecOp<bf16_t> {
  using Op = Op16;
};
template <>
struct DecOp<float> {
  using Op = OpF32;
};

constexpr int DEC_PITCH = 128 + 16;  // bytes of a staged weight row: 128 and one vector of padding

// Row-major weights of SETS x 16 rows, 128 bytes of every row per step. A wave reads eight whole 128-byte lines per
// load (lane / 8 the row, lane % 8 the 16-byte part), puts them into LDS of its own and takes the matrix unit's
// fragments from there (lane % 16 the row, lane / 16 the k): fragments loaded straight from memory would ask
// for 16 half lines per load. Only the wave itself touches its LDS, so there is no barrier in the K loop.
template <typename T, int SETS>
struct RowStep {
  static constexpr int VN = Vec<T>::N;
  static constexpr int STEP = 128 / (int)sizeof(T);  // k per step
  static constexpr int KST = STEP / 32;              // matrix steps of 32 k
  static constexpr int VPF = DecOp<T>::Op::VPF;
  static constexpr int XV = KST * VPF;               // vectors of a column's fragment per step
  static constexpr int LDS_BYTES = SETS * 16 * DEC_PITCH;
  struct Regs {
    u32x4 w[2 * SETS];
  };
  // rows[i]: start of this lane's row of load i
  __device__ __forceinline__ static void load(Regs& r, const T* const (&rows)[2 * SETS], int step, int K, int lane) {
    const int col = min(step * STEP + (lane & 7) * VN, K - VN);
#pragma unroll
    for (int i = 0; i < 2 * SETS; ++i) r.w[i] = ld16_nt(rows[i] + col);
  }
  __device__ __forceinline__ static void stage(const Regs& r, unsigned char* lds, int step, int K, int lane) {
    const bool in = step * STEP + (lane & 7) * VN < K;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 2 * SETS; ++i)
      st16(lds + (i * 8 + (lane >> 3)) * DEC_PITCH + (lane & 7) * 16, in ? r.w[i] : zero);
  }
  __device__ __forceinline__ static void frag(const unsigned char* lds, int set, int kk, int lane, u32x4 (&f)[VPF]) {
    const unsigned char* p = lds + (set * 16 + (lane & 15)) * DEC_PITCH + kk * 32 * (int)sizeof(T) +
                             (lane >> 4) * 8 * (int)sizeof(T);
#pragma unroll
    for (int q = 0; q < VPF; ++q) f[q] = ld16(p + q * 16);
  }
  // this lane's fragments of a column (a row of x or h): k = kk * 32 + (lane / 16) * 8 of the step
  __device__ __forceinline__ static void load_col(u32x4 (&x)[XV], const T* col, int step, int K, int lane) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int kk = 0; kk < KST; ++kk) {
      const int k = step * STEP + kk * 32 + (lane >> 4) * 8;
#pragma unroll
      for (int q = 0; q < VPF; ++q) {
        const u32x4 v = ld16(col + min(k, K - 8) + q * VN);
        x[kk * VPF + q] = k < K ? v : zero;
      }
    }
  }
};

// Packed 4-bit weights of one 16-row block, 128 k per step: one load is a code tile, and a lane's 16 bytes are the
// 32 k of one row that share a scale. The word j of them is its fragment of matrix step j, whose k are
// (lane / 16) * 32 + 8 j on: the columns' fragments follow that order.
struct W4Step {
  static constexpr int STEP = W4_TILE_K;
  static constexpr int XV = 4;
  struct Regs {
    u32x4 w;
    uint32_t s;
  };
  __device__ __forceinline__ static void load(Regs& r, const uint8_t* codes, const uint8_t* scales, int step, int lane) {
    r.w = ld16_nt(codes + (int64_t)step * W4_CODE_TILE + lane * 16);
    r.s = scales[(step >> 2) * W4_SCALE_TILE + lane * 4 + (step & 3)];
  }
  __device__ __forceinline__ static void load_col(u32x4 (&x)[XV], const bf16_t* col, int step, int K, int lane) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int k = step * STEP + (lane >> 4) * 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 v = ld16(col + min(k, K - 32) + 8 * j);
      x[j] = k < K ? v : zero;
    }
  }
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// ------------------------------------------------------------------------------------------------
// gate / up
// ------------------------------------------------------------------------------------------------
// A tile is one expert's 16 columns of h. The eight waves take its K steps in turn and add their sums through LDS
// in wave order.
template <typename T, bool W4, int NB>
struct GateUp {
  using RS = RowStep<T, 2>;
  static constexpr int PF = W4 ? 3 : 3;  // steps of loads in flight per wave
  static constexpr int WAVE_LDS = W4 ? 2 * NB * 4 * 64 * 4 : RS::LDS_BYTES;
  static_assert(WAVE_LDS >= 2 * NB * 4 * 64 * 4, "a wave's sums fit its LDS");
  static constexpr int XV = W4 ? W4Step::XV : RS::XV;

  __device__ __forceinline__ static void tile(const DecodeArgs& a, const Choice& c, int i, int ft, unsigned char* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = a.H, F = a.F, f0 = ft * 16;
    const int64_t l = c.expert[i] % a.El;
    const uint32_t mask = c.mask[i];
    unsigned char* lds = smem + wave * WAVE_LDS;
    // columns of tokens elsewhere read a token of this expert (the same cache lines) and are dropped at the end
    const T* cols[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int t = nb * 16 + (lane & 15);
      cols[nb] = static_cast<const T*>(a.x) + (int64_t)(((mask >> t) & 1u) ? t : __builtin_ctz(mask)) * K;
    }
    f32x4 acc[2][NB];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[s][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

    if constexpr (W4) {
      const int kc = (K + W4_TILE_K - 1) / W4_TILE_K, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
      const int64_t rb = (l * 2 * F + f0) / 16, ub = (l * 2 * F + F + f0) / 16;
      const uint8_t* wc = static_cast<const uint8_t*>(a.w_gu);
      const uint8_t *gc = wc + rb * kc * W4_CODE_TILE, *uc = wc + ub * kc * W4_CODE_TILE;
      const uint8_t *gs = a.s_gu + rb * ks * W4_SCALE_TILE, *us = a.s_gu + ub * ks * W4_SCALE_TILE;
      W4Step::Regs rg[PF], ru[PF];
      u32x4 rx[PF][NB][XV];
      const int last = kc - 1;
      auto load = [&](int st, int u) {
        const int s = min(st, last);
        W4Step::load(rg[u], gc, gs, s, lane);
        W4Step::load(ru[u], uc, us, s, lane);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) W4Step::load_col(rx[u][nb], reinterpret_cast<const bf16_t*>(cols[nb]), s, K, lane);
      };
#pragma unroll
      for (int u = 0; u < PF; ++u) load(wave + u * DEC_NW, u);
      for (int s0 = wave; s0 < kc; s0 += PF * DEC_NW) {
#pragma unroll
        for (int u = 0; u < PF; ++u) {
          const int st = s0 + u * DEC_NW;
          if (st < kc) {
            const float sg = w4_scale(rg[u].s), su = w4_scale(ru[u].s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const u32x4 ag[1] = {w4_to_bf16(rg[u].w[j], sg)}, au[1] = {w4_to_bf16(ru[u].w[j], su)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const u32x4 b[1] = {rx[u][nb][j]};
                Op16::step(acc[0][nb], ag, b);
                Op16::step(acc[1][nb], au, b);
              }
            }
            load(st + PF * DEC_NW, u);
          }
        }
      }
    } else {
      using Op = typename DecOp<T>::Op;
      const T* W = static_cast<const T*>(a.w_gu) + l * 2 * F * K;
      const T* rows[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int f = min(f0 + (q & 1) * 8 + (lane >> 3), F - 1);
        rows[q] = W + (int64_t)((q >> 1) * F + f) * K;
      }
      typename RS::Regs rw[PF];
      u32x4 rx[PF][NB][XV];
      const int ns = (K + RS::STEP - 1) / RS::STEP, last = ns - 1;
      auto load = [&](int st, int u) {
        const int s = min(st, last);
        RS::load(rw[u], rows, s, K, lane);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) RS::load_col(rx[u][nb], cols[nb], s, K, lane);
      };
#pragma unroll
      for (int u = 0; u < PF; ++u) load(wave + u * DEC_NW, u);
      for (int s0 = wave; s0 < ns; s0 += PF * DEC_NW) {
#pragma unroll
        for (int u = 0; u < PF; ++u) {
          const int st = s0 + u * DEC_NW;
          if (st < ns) {
            RS::stage(rw[u], lds, st, K, lane);
#pragma unroll
            for (int kk = 0; kk < RS::KST; ++kk) {
              u32x4 fg[RS::VPF], fu[RS::VPF];
              RS::frag(lds, 0, kk, lane, fg);
              RS::frag(lds, 1, kk, lane, fu);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                u32x4 b[RS::VPF];
#pragma unroll
                for (int q = 0; q < RS::VPF; ++q) b[q] = rx[u][nb][kk * RS::VPF + q];
                Op::step(acc[0][nb], fg, b);
                Op::step(acc[1][nb], fu, b);
              }
            }
            load(st + PF * DEC_NW, u);
          }
        }
      }
    }
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[((s * NB + nb) * 4 + q) * 64 + lane] = acc[s][nb][q];
    __syncthreads();
    for (int o = tid; o < NB * 256; o += DEC_NTH) {
      const int ln = o & 63, q = (o >> 6) & 3, nb = o >> 8;
      const int t = nb * 16 + (ln & 15), f = f0 + (ln >> 4) * 4 + q;
      if (((mask >> t) & 1u) && f < F) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < DEC_NW; ++w) {
          const float* r = reinterpret_cast<const float*>(smem + w * WAVE_LDS);
          g += r[(nb * 4 + q) * 64 + ln];
          u += r[((NB + nb) * 4 + q) * 64 + ln];
        }
        const float h = silu(g) * u;
        const int64_t at = (int64_t)(t * a.k + c.slot[i][t]) * F + f;
        if constexpr (sizeof(T) == 2) {
          const bf16_t hi = (bf16_t)h;
          static_cast<bf16_t*>(a.h)[at] = hi;
          static_cast<bf16_t*>(a.h)[(int64_t)a.T * a.k * F + at] = (bf16_t)(h - (float)hi);
        } else {
          static_cast<float*>(a.h)[at] = h;
        }
      }
    }
    __syncthreads();  // the sums are read before the next tile's stages overwrite them
  }
};

template <typename T, bool W4, int NB>
__global__ __launch_bounds__(DEC_NTH) void decode_gate_up_kernel(DecodeArgs a) {
  using G = GateUp<T, W4, NB>;
  __shared__ Choice c;
  __shared__ __attribute__((aligned(16))) unsigned char smem[DEC_NW * G::WAVE_LDS];
  choose(a, c, blockIdx.x == 0);
  const int nft = (a.F + 15) / 16, total = c.n * nft;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) G::tile(a, c, tile / nft, tile % nft, smem);
}

// ------------------------------------------------------------------------------------------------
// down and combine
// ------------------------------------------------------------------------------------------------
// A tile is 16 columns of y for every token, over all chosen experts. The units (expert, K step), expert by expert,
// are cut into eight runs, one per wave; where a run passes from an expert to the next the wave multiplies its sums by
// the tokens' routing weights and adds them up, and the waves' results are added through LDS in wave order.
// For bf16 layers h has two bf16 parts, hi and lo: h keeps 16 significant bits at the price of a second matrix
// step, which costs nothing next to the weights' bytes.
template <typename T, bool W4, int NB>
struct Down {
  using RS = RowStep<T, 1>;
  static constexpr int PF = W4 ? (NB == 1 ? 3 : 2) : (NB == 1 ? 4 : 3);
  static constexpr int HP = sizeof(T) == 2 ? 2 : 1;  // parts of h
  static constexpr int WAVE_LDS = W4 ? NB * 4 * 64 * 4 : RS::LDS_BYTES;
  static_assert(WAVE_LDS >= NB * 4 * 64 * 4, "a wave's sums fit its LDS");
  static constexpr int XV = W4 ? W4Step::XV : RS::XV;

  __device__ __forceinline__ static void tile(const DecodeArgs& a, const Choice& c, int n0, unsigned char* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = a.F, H = a.H;
    constexpr int STEP = W4 ? W4Step::STEP : RS::STEP;
    const int ns = (K + STEP - 1) / STEP, units = c.n * ns;
    const int per = (units + DEC_NW - 1) / DEC_NW;
    const int u_begin = min(units, wave * per), u_end = min(units, u_begin + per);
    unsigned char* lds = smem + wave * WAVE_LDS;
    const int64_t lo_off = (int64_t)a.T * a.k * K;

    f32x4 acc[NB], y[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[nb] = y[nb] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Slot {
      typename RS::Regs row;
      W4Step::Regs w4;
      u32x4 x[NB][HP][XV];
    };
    Slot buf[PF];
    int li = ns > 0 ? u_begin / ns : 0, ls = u_begin - li * ns;  // the next unit to load
    auto load = [&](int u) {
      const int64_t l = c.expert[li] % a.El;
      const uint32_t mask = c.mask[li];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int tt = nb * 16 + (lane & 15);
        const int t = ((mask >> tt) & 1u) ? tt : __builtin_ctz(mask);
        const T* col = static_cast<const T*>(a.h) + (int64_t)(t * a.k + c.slot[li][t]) * K;
#pragma unroll
        for (int p = 0; p < HP; ++p) {
          if constexpr (W4) W4Step::load_col(buf[u].x[nb][p], reinterpret_cast<const bf16_t*>(col + p * lo_off), ls, K, lane);
          else RS::load_col(buf[u].x[nb][p], col + p * lo_off, ls, K, lane);
        }
      }
      if constexpr (W4) {
        const int kc = ns, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
        const int64_t rb = (l * H + n0) / 16;
        W4Step::load(buf[u].w4, static_cast<const uint8_t*>(a.w_dn) + rb * kc * W4_CODE_TILE,
                     a.s_dn + rb * ks * W4_SCALE_TILE, ls, lane);
      } else {
        const T* rows[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          rows[q] = static_cast<const T*>(a.w_dn) + (l * H + min(n0 + q * 8 + (lane >> 3), H - 1)) * K;
        RS::load(buf[u].row, rows, ls, K, lane);
      }
      if (li * ns + ls + 1 < u_end) {  // past the last unit: the same one again
        if (++ls == ns) {
          ls = 0;
          ++li;
        }
      }
    };
    if (u_begin < u_end) {
#pragma unroll
      for (int u = 0; u < PF; ++u) load(u);
      int ci = u_begin / ns, cs = u_begin - ci * ns;
      for (int n = u_begin; n < u_end; n += PF) {
#pragma unroll
        for (int u = 0; u < PF; ++u) {
          if (n + u < u_end) {
            if constexpr (W4) {
              const float sc = w4_scale(buf[u].w4.s);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const u32x4 f[1] = {w4_to_bf16(buf[u].w4.w[j], sc)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int p = 0; p < HP; ++p) {
                    const u32x4 b[1] = {buf[u].x[nb][p][j]};
                    Op16::step(acc[nb], f, b);
                  }
              }
            } else {
              RS::stage(buf[u].row, lds, cs, K, lane);
#pragma unroll
              for (int kk = 0; kk < RS::KST; ++kk) {
                u32x4 f[RS::VPF];
                RS::frag(lds, 0, kk, lane, f);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int p = 0; p < HP; ++p) {
                    u32x4 b[RS::VPF];
#pragma unroll
                    for (int q = 0; q < RS::VPF; ++q) b[q] = buf[u].x[nb][p][kk * RS::VPF + q];
                    DecOp<T>::Op::step(acc[nb], f, b);
                  }
              }
            }
            load(u);
            if (++cs == ns || n + u + 1 == u_end) {
              const uint32_t mask = c.mask[ci];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const int t = nb * 16 + (lane & 15);
                const bool on = (mask >> t) & 1u;
                const float w = on ? c.w[t * a.k + c.slot[ci][t]] : 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  y[nb][q] = on ? fmaf(w, acc[nb][q], y[nb][q]) : y[nb][q];
                  acc[nb][q] = 0.f;
                }
              }
              cs = 0;
              ++ci;
            }
          }
        }
      }
    }
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[(nb * 4 + q) * 64 + lane] = y[nb][q];
    __syncthreads();
    for (int o = tid; o < NB * 256; o += DEC_NTH) {
      const int r = o & 15, t = o >> 4;  // 16 threads write 16 columns of one token
      const int nb = t >> 4, q = r & 3, ln = (r >> 2) * 16 + (t & 15);
      if (t < a.T && n0 + r < H) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < DEC_NW; ++w)
          v += reinterpret_cast<const float*>(smem + w * WAVE_LDS)[(nb * 4 + q) * 64 + ln];
        static_cast<T*>(a.y)[(int64_t)t * H + n0 + r] = from_f32<T>(v);
      }
    }
    __syncthreads();
  }
};

template <typename T, bool W4, int NB>
__global__ __launch_bounds__(DEC_NTH) void decode_down_kernel(DecodeArgs a) {
  using D = Down<T, W4, NB>;
  __shared__ Choice c;
  __shared__ __attribute__((aligned(16))) unsigned char smem[DEC_NW * D::WAVE_LDS];
  choose(a, c, false);
  const int total = (a.H + 15) / 16;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) D::tile(a, c, tile * 16, smem);
}

template <typename T>
void launch_route_rows(const T* x, const float* w, const float* bias, int64_t bias_stride, int T_, int H, int E,
                       float* logits, hipStream_t stream) {
  auto go = [&](auto tb) {
    constexpr int TB = decltype(tb)::value;
    decode_route_kernel<T, TB><<<dim3(E, ceil_div_host(T_, TB)), 256, 0, stream>>>(x, w, bias, bias_stride, T_, H, E,
                                                                                   logits);
  };
  if (T_ == 1) go(std::integral_constant<int, 1>{});
  else if (T_ <= 2) go(std::integral_constant<int, 2>{});
  else if (T_ <= 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
}

template <typename T, bool W4, int NB>
void launch_experts(const DecodeArgs& a, int num_cus, hipStream_t stream) {
  const int pairs = std::min(a.T * a.k, a.E);
  const int64_t gu = (int64_t)pairs * ((a.F + 15) / 16);
  decode_gate_up_kernel<T, W4, NB><<<(int)std::min<int64_t>(gu, 2 * num_cus), DEC_NTH, 0, stream>>>(a);
  decode_down_kernel<T, W4, NB><<<std::min((a.H + 15) / 16, 2 * num_cus), DEC_NTH, 0, stream>>>(a);
}

}  // namespace

size_t decode_workspace_bytes(int T, int k, int F) { return align256((size_t)T * k * (size_t)F * 4); }

hipError_t launch_layer_decode(const DecodeCall& d, int num_cus, hipStream_t stream) {
  if (d.bf16)
    launch_route_rows(static_cast<const bf16_t*>(d.x), d.w_router, d.bias, d.bias_stride, d.T, d.H, d.E, d.logits, stream);
  else
    launch_route_rows(static_cast<const float*>(d.x), d.w_router, d.bias, d.bias_stride, d.T, d.H, d.E, d.logits, stream);
  DecodeArgs a{};
  a.x = d.x;
  a.logits = d.logits;
  a.T = d.T;
  a.H = d.H;
  a.E = d.E;
  a.El = d.E / d.R;
  a.k = d.k;
  a.C = d.C;
  a.F = d.F;
  a.w_gu = d.w_gu;
  a.w_dn = d.w_dn;
  a.s_gu = d.s_gu;
  a.s_dn = d.s_dn;
  a.ids = d.ids;
  a.wts = d.wts;
  a.y = d.y;
  a.h = d.workspace;
  const bool two = d.T > 16;
  if (!d.bf16) two ? launch_experts<float, false, 2>(a, num_cus, stream) : launch_experts<float, false, 1>(a, num_cus, stream);
  else if (d.s_gu) two ? launch_experts<bf16_t, true, 2>(a, num_cus, stream) : launch_experts<bf16_t, true, 1>(a, num_cus, stream);
  else two ? launch_experts<bf16_t, false, 2>(a, num_cus, stream) : launch_experts<bf16_t, false, 1>(a, num_cus, stream);
  return hipGetLastError();
}

}  // namespace moe
