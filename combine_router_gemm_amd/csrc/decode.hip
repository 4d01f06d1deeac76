// The whole MoE layer for a few tokens (T <= 32): moe_layer_decode and moe_layer_decode_w4.
//
//   logits = x Wr^T + b            decode_route_kernel
//   top-k, softmax, capacity       choose(), by every workgroup of the next kernel for itself
//   h = silu(x Wg^T) * (x Wu^T)    decode_gate_up_kernel, per chosen expert
//   y = sum_j w_j h_j Wd^T         decode_down_kernel
//
// What bounds it: the bytes of the chosen experts' weights, each read once. The weights are the M operand of the
// matrix unit (16 output columns per tile) and an expert's tokens its N operand, gathered by the loads. No partial
// result is added atomically: the down kernel adds a token's experts in expert order, and where an H of few tiles has
// it split, decode_sum_kernel adds the parts in theirs.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "mfma.h"
#include "topk.h"
#include "w4.h"

namespace moe {

namespace {

constexpr int DEC_GU_NW = 8;  // waves of a gate/up workgroup: they split K
constexpr int DEC_PAIRS = MOE_DECODE_MAX_TOKENS * MOE_MAX_TOPK;

struct Choice;

struct DecodeArgs {
  const void* x;        // [T, H]; with 4-bit weights rows of w4_pitch(H), each 128 k in w4_place order
  const float* logits;  // [T, E]
  int T, H, E, El, k, C, F;
  const void* w_gu;     // [El, 2F, H], or its packed codes
  const void* w_dn;     // [El, H, F]
  const uint8_t* s_gu;  // scales of packed weights
  const uint8_t* s_dn;
  int* ids;             // [T, k]
  float* wts;           // [T, k]
  void* y;              // [T, H]
  Choice* choice;       // written by the gate/up kernel, read by the down kernel
  void* h;              // [T * k, F] by row of Choice: fp32, or for bf16 layers the bf16 nearest to h and then
                        // [T * k, F] its remainder; with 4-bit weights rows of both parts, at w4_place2
  float* partial;       // [split, T, H] sums of the down kernel's parts, where it is split
  int split;
};

// With 4-bit weights the matrix step j of 128 k takes k = 32 g + 8 j .. + 7 from lane group g (W4Step). Rows of x and h
// are kept with those four pieces of a step side by side, so that a row's fragment load is one 64-byte segment rather
// than four pieces of 16 bytes 64 apart: element k of a row is at w4_place(k). The router writes x so, gate/up h.
__host__ __device__ __forceinline__ int w4_pitch(int K) { return (K + W4_TILE_K - 1) / W4_TILE_K * W4_TILE_K; }
__device__ __forceinline__ int w4_place(int k) {
  return (k & ~(W4_TILE_K - 1)) + ((k >> 3) & 3) * 32 + ((k >> 5) & 3) * 8 + (k & 7);
}
// the same for the first of h's two parts, each 32 elements of it followed by those of the second
__device__ __forceinline__ int w4_place2(int k) { return w4_place(k) * 2 - (((k >> 5) & 3) * 8 + (k & 7)); }

// ------------------------------------------------------------------------------------------------
// router
// ------------------------------------------------------------------------------------------------
// One workgroup per EB experts and TB tokens: its 256 threads share the fp32 weight rows, every thread takes eight
// consecutive k at a time (exact products, at most ceil(H / 2048) * 8 fp32 additions in a row), then a fixed
// tree of additions. Bound by the reads of x and the weights from L2: EB experts share one read of x.
template <typename T>
__device__ __forceinline__ void unpack8(const u32x4 (&v)[sizeof(T) / 2], float (&o)[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack(v[0], o);
  } else {
    unpack(v[0], *reinterpret_cast<float(*)[4]>(&o[0]));
    unpack(v[1], *reinterpret_cast<float(*)[4]>(&o[4]));
  }
}

template <typename T, int TB, int EB>
__global__ __launch_bounds__(256) void decode_route_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                                           const float* __restrict__ bias, int64_t bias_stride, int T_,
                                                           int H, int E, float* __restrict__ logits,
                                                           bf16_t* __restrict__ placed) {
  __shared__ float s_sum[4][EB][TB];
  const int e0 = blockIdx.x * EB, t0 = blockIdx.y * TB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float acc[EB][TB];
#pragma unroll
  for (int i = 0; i < EB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = 0.f;
  constexpr int XV = (int)sizeof(T) / 2;  // 16-byte vectors of eight elements
  for (int c = tid * 8; c < H; c += 2048) {
    u32x4 wr[EB][2], xr[TB][XV];
#pragma unroll
    for (int i = 0; i < EB; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) wr[i][q] = ld16(w + (int64_t)min(e0 + i, E - 1) * H + c + 4 * q);
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int q = 0; q < XV; ++q) xr[j][q] = ld16(x + (int64_t)min(t0 + j, T_ - 1) * H + c + Vec<T>::N * q);
    __builtin_amdgcn_sched_barrier(0);  // all requested before the first is waited for
    float wv[EB][8];
#pragma unroll
    for (int i = 0; i < EB; ++i) unpack8<float>(wr[i], wv[i]);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      float xv[8];
      unpack8<T>(xr[j], xv);
#pragma unroll
      for (int i = 0; i < EB; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i][j] = fmaf(xv[q], wv[i][q], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < EB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const float s = wave_sum(acc[i][j]);
      if (lane == 0) s_sum[wave][i][j] = s;
    }
  __syncthreads();
  if constexpr (sizeof(T) == 2) {
    if (placed) {  // x in w4_place order, by all workgroups together
      const int n = min(TB, T_ - t0) * (H / 8);
      for (int c = blockIdx.x * 256 + tid; c < n; c += gridDim.x * 256) {
        const int t = t0 + c / (H / 8), k = c % (H / 8) * 8;
        st16(placed + (int64_t)t * w4_pitch(H) + w4_place(k), ld16(x + (int64_t)t * H + k));
      }
    }
  }
  if (tid < EB * TB) {
    const int i = tid / TB, j = tid % TB, e = e0 + i, t = t0 + j;
    if (e < E && t < T_) {
      float v = (s_sum[0][i][j] + s_sum[1][i][j]) + (s_sum[2][i][j] + s_sum[3][i][j]);
      if (bias) v += bias[(int64_t)t * bias_stride + e];
      logits[(int64_t)t * E + e] = v;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// choice of experts
// ------------------------------------------------------------------------------------------------
// The kept pairs by local expert. Two experts of different ranks that share a weight set (e mod El) are one entry,
// and a token that chose both is one row with the sum of its weights: h and the expert's output are the same.
struct Choice {
  int n;                           // local experts with a row, ascending
  int expert[DEC_PAIRS];
  int row0[DEC_PAIRS + 1];         // its rows (tokens ascending): row0[i] .. row0[i + 1]
  float w[DEC_PAIRS];              // routing weight of a row
  int token[DEC_PAIRS];            // token of a row
};
struct ChoiceScratch {
  int wcnt[DEC_GU_NW], wrow[DEC_GU_NW];
  int ids[DEC_PAIRS], local_id[DEC_PAIRS];
  float pw[DEC_PAIRS];
  uint32_t chosen[MOE_MAX_EXPERTS];  // tokens of a (global) expert, then those within its capacity
  uint32_t local[MOE_MAX_EXPERTS];   // tokens of a local expert
  uint16_t place[MOE_MAX_EXPERTS];
};

// Top-k, softmax and capacity of every token from the logits, by a whole workgroup: a wave per token (TW of them
// interleaved: a round is one long chain of dependent operations), expert lane * V + i in the lane's i-th value; each
// of the k rounds takes the wave's largest key, the lowest expert among equals (moe_route's rule: -0 == +0, a NaN ranks
// as -inf). Every gate/up workgroup does it for itself (one token 4-6 us of which 1.2 are the logits' latency): one
// that did it for all would have to be waited for. Workgroup 0 publishes the result for the down kernel.
template <int TW>
__device__ __forceinline__ void choose_topk(const DecodeArgs& a, ChoiceScratch& c, int t0, bool write) {
  constexpr int VMAX = MOE_MAX_EXPERTS / 64;
  const int lane = threadIdx.x & 63;
  const int V = (a.E + 63) / 64;
  // every logit requested at once; a lane without an i-th expert, and a token past T, read the last one
  float v[TW][VMAX];
#pragma unroll
  for (int x = 0; x < TW; ++x)
#pragma unroll
    for (int i = 0; i < VMAX; ++i)
      v[x][i] = i < V ? a.logits[(int64_t)min(t0 + x * DEC_GU_NW, a.T - 1) * a.E + min(lane * V + i, a.E - 1)] : 0.f;
  int key[TW][VMAX];
#pragma unroll
  for (int x = 0; x < TW; ++x)
#pragma unroll
    for (int i = 0; i < VMAX; ++i) {
      const float s = v[x][i] + 0.0f;  // -0 -> +0
      key[x][i] = i < V && lane * V + i < a.E ? float_key(s == s ? s : -INFINITY) : INT_MIN;
    }
  // lane j ends up with the j-th selection. The rounds are a loop and not unrolled: every workgroup runs them once, so
  // straight code is paid for in instruction fetches (f32 layer of 8 experts, one token: the kernel 6.5 -> 5.9 us)
  float mine_v[TW], top[TW];
  int mine[TW];
#pragma unroll
  for (int x = 0; x < TW; ++x) {
    mine_v[x] = top[x] = 0.f;
    mine[x] = 0;
  }
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
#pragma unroll
    for (int x = 0; x < TW; ++x) {
      int head = key[x][0], at = 0;
#pragma unroll
      for (int i = 1; i < VMAX; ++i) {
        at = key[x][i] > head ? i : at;
        head = max(head, key[x][i]);
      }
      const int m = wave_max_i32(head);
      const int wl = __builtin_ctzll(__ballot(head == m));  // k <= E: m is a present value's key
      const int e = __builtin_amdgcn_readlane(lane * V + at, wl);
      top[x] = j == 0 ? key_float(m) : top[x];
      mine_v[x] = lane == j ? key_float(m) : mine_v[x];
      mine[x] = lane == j ? e : mine[x];
      const int gone = lane == wl ? at : VMAX;
#pragma unroll
      for (int i = 0; i < VMAX; ++i) key[x][i] = i == gone ? INT_MIN : key[x][i];
    }
  }
#pragma unroll
  for (int x = 0; x < TW; ++x) {
    const int t = t0 + x * DEC_GU_NW;
    const float z = lane < a.k ? expf(mine_v[x] - top[x]) : 0.f;
    const float w = z / wave_sum(z);
    if (lane < a.k && t < a.T) {
      const int p = t * a.k + lane;
      c.ids[p] = mine[x];
      c.local_id[p] = mine[x] % a.El;
      c.pw[p] = w;
      atomicOr(&c.chosen[mine[x]], 1u << t);
      if (write) {
        a.ids[p] = mine[x];
        a.wts[p] = w;
      }
    }
  }
}

__device__ __forceinline__ void choose(const DecodeArgs& a, Choice& o, ChoiceScratch& c, bool write) {
  constexpr int NW = DEC_GU_NW, NTH = NW * 64;
  static_assert(NTH >= MOE_MAX_EXPERTS && NTH >= DEC_PAIRS, "a thread per expert and per pair");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  c.chosen[tid] = 0;
  c.local[tid] = 0;
  __syncthreads();
  if (a.T <= NW) {
    if (wave < a.T) choose_topk<1>(a, c, wave, write);
  } else {
    for (int t0 = wave; t0 < a.T; t0 += 2 * NW) choose_topk<2>(a, c, t0, write);
  }
  __syncthreads();
  // the first C tokens of every expert
  if (tid < a.E) {
    uint32_t m = c.chosen[tid];
    for (int over = __popc(m) - a.C; over > 0; --over) m &= ~(0x80000000u >> __clz(m));
    c.chosen[tid] = m;
    if (m != 0) atomicOr(&c.local[tid % a.El], m);
  }
  __syncthreads();
  // local experts with any, and their rows: exclusive scans over the threads
  const uint32_t m = tid < a.El ? c.local[tid] : 0u;
  const uint64_t b = __ballot(m != 0);
  int rows = __popc(m);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(rows, off, 64);
    if (lane >= off) rows += v;
  }
  if (lane == 63) {
    c.wcnt[wave] = __popcll(b);
    c.wrow[wave] = rows;
  }
  __syncthreads();
  int i = __popcll(b & lanemask_lt()), row = rows - __popc(m);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    i += w < wave ? c.wcnt[w] : 0;
    row += w < wave ? c.wrow[w] : 0;
  }
  if (m != 0) {
    o.expert[i] = tid;
    o.row0[i] = row;
    c.place[tid] = (uint16_t)i;
  }
  if (tid == NTH - 1) {  // past the last expert: the totals
    o.n = i + (m != 0);
    o.row0[i + (m != 0)] = row + __popc(m);
  }
  __syncthreads();
  // the first slot of a token that reaches a local expert writes its row, with the weights of the later ones added
  if (tid < a.T * a.k) {
    const int t = tid / a.k, p0 = t * a.k, le = c.local_id[tid];
    float w = 0.f;
    bool first = true, mine = false;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      const bool on = c.local_id[p0 + j] == le && ((c.chosen[c.ids[p0 + j]] >> t) & 1u);
      w += on && p0 + j >= tid ? c.pw[p0 + j] : 0.f;
      first = first && !(on && p0 + j < tid);
      mine = mine || (on && p0 + j == tid);
    }
    if (first && mine) {
      const int r = o.row0[c.place[le]] + __popc(c.local[le] & ((1u << t) - 1u));
      o.token[r] = t;
      o.w[r] = w;
    }
  }
  __syncthreads();
  if (write)
    for (int x = tid; x < (int)(sizeof(Choice) / 4); x += NTH)
      reinterpret_cast<int*>(a.choice)[x] = reinterpret_cast<const int*>(&o)[x];
}

// ------------------------------------------------------------------------------------------------
// operands
// ------------------------------------------------------------------------------------------------
template <typename T>
struct DecOp;
template <>
struct DecOp<bf16_t> {
  static constexpr int VPF = Op16::VPF;
  static __device__ __forceinline__ void step(f32x4& acc, const u32x4 (&a)[1], const u32x4 (&b)[1]) {
    Op16::step(acc, a, b);
  }
};
// f32: the eight products of a step are summed apart and then added, so that the roundings of a long K stay those of
// K / 256 additions per wave rather than of K / 32 (y is off by 3.6e-7 of its norm at H 4096, F 14336)
template <>
struct DecOp<float> {
  static constexpr int VPF = OpF32::VPF;
  static __device__ __forceinline__ void step(f32x4& acc, const u32x4 (&a)[2], const u32x4 (&b)[2]) {
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
    OpF32::step(part, a, b);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] += part[q];
  }
};

// Columns (rows of x or h) are read with buffer loads: a lane without one, or past K, reads at an offset beyond the
// buffer, which the hardware answers with zeros and without a memory request.
constexpr int DEC_NONE = 0x7ffff000;
constexpr int DEC_COL_MAX = 3 * 64 * 2;  // the most that is added to it: the fourth step of h's two parts (W4Step)
static_assert((int64_t)DEC_NONE + DEC_COL_MAX + 16 <= INT32_MAX, "offsets are signed 32-bit sums");
static_assert((int64_t)MOE_DECODE_MAX_TOKENS * kDecodeMaxH * 4 <= DEC_NONE &&
                  (int64_t)(MOE_DECODE_MAX_TOKENS * MOE_MAX_TOPK + MOE_DECODE_MAX_TOKENS) * kDecodeMaxF * 4 <= DEC_NONE,
              "past the end of the rows of x and of both parts of h");
__device__ __forceinline__ u32x4 ld_col(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

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
  static constexpr int VPF = DecOp<T>::VPF;
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
  // this lane's fragments of a column (a row of x or h, at byte `row` of the buffer): k = kk * 32 + (lane / 16) * 8
  __device__ __forceinline__ static void load_col(u32x4 (&x)[XV], __amdgpu_buffer_rsrc_t r, int row, int step, int K,
                                                  int lane) {
#pragma unroll
    for (int kk = 0; kk < KST; ++kk) {
      const int k = step * STEP + kk * 32 + (lane >> 4) * 8;
      const int off = row >= 0 && k < K ? row + k * (int)sizeof(T) : DEC_NONE;
#pragma unroll
      for (int q = 0; q < VPF; ++q) x[kk * VPF + q] = ld_col(r, off + q * 16);
    }
  }
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Packed 4-bit weights of BL 16-row blocks, 128 k per step. One load is a code tile, and a lane's 16 bytes are the 32
// k of one row that share a scale. The word j of them is its fragment of matrix step j, whose k are (lane / 16) * 32
// + 8 j on: the columns' fragments follow that order. A load of a byte per lane takes as long as one of sixteen, so
// scales come sixteen bytes per lane, four tiles at a time, through LDS of the wave's own, and several blocks share a
// column's fragments. Where only four columns are in use (CW 4, not 16) one load takes what four would: lane c of 16
// takes column c % 4's fragment of step c / 4, and a rotation within the 16 lanes brings it to its column when that
// step comes. What then stands in the other columns is never looked at. One token of a DeepSeek-V3 share: down 17.0 ->
// 15.7 us, and gate/up has registers for a third step in flight; eight columns in two loads gave nothing (Kimi-K2
// share, 32 tokens).
template <int BL>
struct W4Step {
  static constexpr int STEP = W4_TILE_K;
  static constexpr int CHUNK = 4;  // scale tiles in LDS: 2048 k
  static constexpr int LDS_BYTES = BL * CHUNK * W4_SCALE_TILE;
  // the blocks' tiles: wave-uniform, so that they stay in scalar registers
  const uint8_t* codes[BL];
  const uint8_t* scales[BL];
  __device__ __forceinline__ void block(int b, const void* c, const uint8_t* s, int64_t rb, int K) {
    codes[b] = static_cast<const uint8_t*>(c) + rb * ((K + W4_TILE_K - 1) / W4_TILE_K) * W4_CODE_TILE;
    scales[b] = s + rb * ((K + W4_STILE_K - 1) / W4_STILE_K) * W4_SCALE_TILE;
  }
  __device__ __forceinline__ void load(u32x4 (&w)[BL], int step, int lane) const {
#pragma unroll
    for (int b = 0; b < BL; ++b) w[b] = ld16_nt(codes[b] + (int64_t)step * W4_CODE_TILE + (uint32_t)(lane * 16));
  }
  // scale tiles t0 .. t0 + CHUNK - 1 (of ks) to LDS, through registers
  __device__ __forceinline__ void load_scales(u32x4 (&v)[BL], int t0, int ks, int lane) const {
#pragma unroll
    for (int b = 0; b < BL; ++b)
      v[b] = ld16(scales[b] + (uint32_t)(min(t0 + (lane >> 4), ks - 1) * W4_SCALE_TILE + (lane & 15) * 16));
  }
  __device__ __forceinline__ static void store_scales(const u32x4 (&v)[BL], unsigned char* lds, int lane) {
#pragma unroll
    for (int b = 0; b < BL; ++b) st16(lds + b * CHUNK * W4_SCALE_TILE + lane * 16, v[b]);
  }
  __device__ __forceinline__ static float scale(const unsigned char* lds, int b, int t0, int step, int lane) {
    return w4_scale(lds[(b * CHUNK + (step >> 2) - t0) * W4_SCALE_TILE + lane * 4 + (step & 3)]);
  }
  // row: byte of the buffer where the row of this lane's column starts (lane % 16 % CW), or -1
  template <int PARTS, int CW>
  __device__ __forceinline__ static void load_col(u32x4 (&x)[CW / 4], __amdgpu_buffer_rsrc_t r, int row, int step, int K,
                                                  int lane) {
    const bool in = row >= 0 && step * STEP + (lane >> 4) * 32 < K;
    const int off =
        in ? row + step * (STEP * 2 * PARTS) + (lane >> 4) * 16 + (lane & 15) / CW * (64 * PARTS) : DEC_NONE;
#pragma unroll
    for (int q = 0; q < CW / 4; ++q) {
      static_assert((CW / 4 - 1) * 64 * PARTS <= DEC_COL_MAX, "");
      x[q] = ld_col(r, off + q * (64 * PARTS));
    }
  }
  // the fragments of matrix step j
  template <int CW>
  __device__ __forceinline__ static u32x4 col(const u32x4 (&x)[CW / 4], int j) {
    if constexpr (CW == 16) {
      return x[j];
    } else {
      const u32x4 v = x[0];
      switch (j) {  // lane c from lane c + 4 j: a rotation to the right by 16 less that
        case 1: return u32x4{dpp_u32<0x12c>(v.x), dpp_u32<0x12c>(v.y), dpp_u32<0x12c>(v.z), dpp_u32<0x12c>(v.w)};
        case 2: return u32x4{dpp_u32<0x128>(v.x), dpp_u32<0x128>(v.y), dpp_u32<0x128>(v.z), dpp_u32<0x128>(v.w)};
        case 3: return u32x4{dpp_u32<0x124>(v.x), dpp_u32<0x124>(v.y), dpp_u32<0x124>(v.z), dpp_u32<0x124>(v.w)};
        default: return v;
      }
    }
  }
};

// Steps s, s + D, ... below stop through PF slots of registers, whose first loads are under way: use(st, u) a step
// from slot u, load(st, u) one into it. No load is issued past the end: runs are short (7 to 45 steps), and loads
// that repeat the last step to keep one loop body take as long as the others (gate/up and down, us:
// 16 tokens of a Kimi-K2 share in bf16 349 -> 333 and 198 -> 187; one token of a DeepSeek-V3 share in 4 bits 25.1 ->
// 23.6 and 16.0 -> 12.8).
template <int PF, int D, typename Use, typename Load>
__device__ __forceinline__ void pipeline(int s, int stop, Use use, Load load) {
  for (; s + (2 * PF - 1) * D < stop; s += PF * D) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      use(s + u * D, u);
      load(s + (u + PF) * D, u);
    }
  }
#pragma unroll
  for (int u = 0; u < PF; ++u)
    if (s + u * D < stop) {
      use(s + u * D, u);
      if (s + (u + PF) * D < stop) load(s + (u + PF) * D, u);
    }
#pragma unroll
  for (int u = 0; u < PF - 1; ++u)
    if (s + (u + PF) * D < stop) use(s + (u + PF) * D, u);
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// ------------------------------------------------------------------------------------------------
// gate / up
// ------------------------------------------------------------------------------------------------
// Row-major weights: a tile is 16 columns of h for NB blocks of 16 rows of one expert (two for more than 16 tokens).
// The eight waves split its K and add their sums through LDS in wave order; the next tile's first loads are requested
// before that, so the weight stream does not stop at a tile's end (Mixtral layer, one token, 79.8 -> 77.9 us). The f32
// kernel of two blocks has registers for one step of loads in flight; two spill (whole layer of 32 tokens, 37 experts,
// H 968, F 4992: 507 us against 425).
template <typename T, int NB>
struct GateUp {
  static constexpr int NW = DEC_GU_NW, NTH = NW * 64;
  using RS = RowStep<T, 2>;
  static constexpr int COLS = 16;
  static constexpr int PF = NB == 1 ? 3 : sizeof(T) == 2 ? 2 : 1;  // steps of loads in flight per wave
  static constexpr int RED = 2 * NB * 4 * 64 * 4;
  static constexpr int WAVE_LDS = RED > RS::LDS_BYTES ? RED : RS::LDS_BYTES;

  __device__ __forceinline__ static void run(const DecodeArgs& a, const Choice& c, unsigned char* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = a.H, F = a.F;
    const int nft = (F + COLS - 1) / COLS, total = c.n * nft;
    unsigned char* lds = smem + wave * WAVE_LDS;
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc((void*)a.x, (short)0, a.T * K * (int)sizeof(T), 0x00020000);
    const int ns = (K + RS::STEP - 1) / RS::STEP;

    // the tile whose loads are requested next
    int tile = blockIdx.x, row0 = 0, cnt = 0, f0 = 0;
    int cols[NB];
    const T* rows[4];
    typename RS::Regs rw[PF];
    u32x4 rx[PF][NB][RS::XV];
    auto load = [&](int st, int u) {
      const int s = min(st, ns - 1);
      RS::load(rw[u], rows, s, K, lane);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) RS::load_col(rx[u][nb], xr, cols[nb], s, K, lane);
    };
    auto start = [&]() {  // the tile's addresses and its first loads
      const int i = tile / nft;
      f0 = (tile - i * nft) * COLS;
      const int64_t l = __builtin_amdgcn_readfirstlane(c.expert[i]);
      row0 = __builtin_amdgcn_readfirstlane(c.row0[i]);
      cnt = __builtin_amdgcn_readfirstlane(c.row0[i + 1]) - row0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int r = nb * 16 + (lane & 15);
        cols[nb] = r < cnt ? c.token[row0 + r] * K * (int)sizeof(T) : -1;
      }
      const T* W = static_cast<const T*>(a.w_gu) + l * 2 * F * K;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int f = min(f0 + (q & 1) * 8 + (lane >> 3), F - 1);
        rows[q] = W + (int64_t)((q >> 1) * F + f) * K;
      }
#pragma unroll
      for (int u = 0; u < PF; ++u) load(wave + u * NW, u);
    };
    if (tile < total) start();
    while (tile < total) {
      f32x4 acc[2][NB];  // gate, up
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[s][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto use = [&](int st, int u) {
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
            DecOp<T>::step(acc[0][nb], fg, b);
            DecOp<T>::step(acc[1][nb], fu, b);
          }
        }
      };
      pipeline<PF, NW>(wave, ns, use, load);
      float* red = reinterpret_cast<float*>(lds);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int q = 0; q < 4; ++q) red[((s * NB + nb) * 4 + q) * 64 + lane] = acc[s][nb][q];
      const int done_row0 = row0, done_cnt = cnt, done_f0 = f0;
      tile += gridDim.x;
      if (tile < total) start();
      lds_barrier();
      for (int o = tid; o < NB * 256; o += NTH) {
        const int ln = o & 63, q = (o >> 6) & 3, nb = o >> 8;
        const int r = nb * 16 + (ln & 15), f = done_f0 + (ln >> 4) * 4 + q;
        if (r < done_cnt && f < F) {
          float g = 0.f, u = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const float* red_w = reinterpret_cast<const float*>(smem + w * WAVE_LDS);
            g += red_w[(nb * 4 + q) * 64 + ln];
            u += red_w[((NB + nb) * 4 + q) * 64 + ln];
          }
          const float h = silu(g) * u;
          const int64_t at = (int64_t)(done_row0 + r) * F + f;
          if constexpr (sizeof(T) == 2) {
            static_cast<bf16_t*>(a.h)[at] = (bf16_t)h;
            static_cast<bf16_t*>(a.h)[at + (int64_t)a.T * a.k * F] = (bf16_t)bf16_rest(h);
          } else {
            static_cast<float*>(a.h)[at] = h;
          }
        }
      }
      lds_barrier();  // the sums are read before the next tile's stages overwrite them
    }
  }
};

// 4-bit weights: a tile is 32 columns of h for all rows of one expert. More than 16 rows take two blocks of columns with
// one step of loads in flight instead of two, and their scales are stored before the columns are loaded: no more
// registers are left with two workgroups per CU, and a spilled one is reloaded behind every load in flight (32 tokens of
// a Kimi-K2 share, some of whose experts have that many rows: 157.5 us with the codes read twice, 145.8 so).
// Each wave takes a run of K, because scales come by four steps. The eight waves share a tile's K, or four, two or one
// of them do where that leaves a wave fewer than seven steps, so that it spends its time on filling and draining its
// loads, and there are tiles enough for every workgroup.
// Whole layers (us, eight always and by this rule): 16 tokens, 64 experts, k 4, H 1024, F 4096 93 -> 67; 32 tokens, 128
// experts, k 8, H 2048, F 768 86 -> 79; 8 tokens, 8 experts, k 2, H 2048, F 8192 46 -> 43. With four steps for seven the
// second took 85.
// ANY_KW: the kernel that can do so; a launch of too few tiles takes the other, 0.5 us faster for one token.
template <bool ANY_KW>
struct GateUpW4 {
  static constexpr int NW = DEC_GU_NW, NTH = NW * 64;
  static constexpr int COLS = 32;
  static constexpr int NBMAX = MOE_DECODE_MAX_TOKENS / 16;
  using WS = W4Step<4>;  // gate, gate, up, up
  static constexpr int RED = 4 * NBMAX * 4 * 64 * 4;
  static constexpr int WAVE_LDS = RED > WS::LDS_BYTES ? RED : WS::LDS_BYTES;
  static constexpr int LW = 3, MIN_STEPS = 7;
  static_assert(NW == 1 << LW, "");
  // whether half of 2^lw waves are better for each of `total` tiles of ns steps
  __host__ __device__ static constexpr bool narrow(int ns, int64_t total, int grid, int lw) {
    return ns < (MIN_STEPS << lw) && (total << lw) / 2 >= (int64_t)NW * grid;
  }

  // K of one tile for kw waves, this one the wk-th; its sums to its LDS
  template <int CW, int NB>
  __device__ __forceinline__ static void multiply(const DecodeArgs& a, const Choice& c, int i, int f0, int kw, int wk,
                                                  unsigned char* lds) {
    // steps of loads in flight per wave, as the registers allow; two for four columns: 22.9 -> 23.6 us (one token,
    // DeepSeek-V3 share), 140 -> 147 us (32 tokens, Kimi-K2 share)
    constexpr int PF = NB == 2 ? 1 : CW == 4 ? 3 : 2;
    const int lane = threadIdx.x & 63;
    const int K = a.H, F = a.F, pitch = w4_pitch(K);
    const int64_t l = __builtin_amdgcn_readfirstlane(c.expert[i]);
    const int row0 = __builtin_amdgcn_readfirstlane(c.row0[i]);
    const int cnt = __builtin_amdgcn_readfirstlane(c.row0[i + 1]) - row0;
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc((void*)a.x, (short)0, a.T * pitch * 2, 0x00020000);
    int cols[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 16 + (lane & 15) % CW;
      cols[nb] = r < cnt ? c.token[row0 + r] * pitch * 2 : -1;
    }
    const int ns = pitch / WS::STEP, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
    const int per = (ns + kw - 1) / kw, begin = wk * per, end = min(ns, begin + per);
    WS ws;
#pragma unroll
    for (int b = 0; b < 4; ++b) ws.block(b, a.w_gu, a.s_gu, (l * 2 * F + (b >> 1) * F + f0) / 16 + (b & 1), K);
    f32x4 acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[nb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 rw[PF][4], rx[PF][NB][CW / 4];
    auto load = [&](int st, int u) {
      const int s = min(st, end - 1);
      ws.load(rw[u], s, lane);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) WS::template load_col<1, CW>(rx[u][nb], xr, cols[nb], s, K, lane);
    };
    for (int s0 = begin; s0 < end;) {
      const int t0 = s0 >> 2, stop = min(end, (t0 + WS::CHUNK) * 4);
      u32x4 sv[4];
      ws.load_scales(sv, t0, ks, lane);
      if (NB > 1) {  // the scales' registers are needed for the columns
        WS::store_scales(sv, lds, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int u = 0; u < PF; ++u) load(s0 + u, u);
      if (NB == 1) WS::store_scales(sv, lds, lane);
      auto use = [&](int st, int u) {
        float sc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) sc[b] = WS::scale(lds, b, t0, st, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4 x[NB][1];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) x[nb][0] = WS::template col<CW>(rx[u][nb], j);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const u32x4 f[1] = {w4_to_bf16(rw[u][b][j], sc[b])};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) Op16::step(acc[nb][b], f, x[nb]);
          }
        }
      };
      pipeline<PF, 1>(s0, stop, use, load);
      s0 = stop;
    }
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[((nb * 4 + b) * 4 + q) * 64 + lane] = acc[nb][b][q];
  }

  // h of one tile from the sums of kw waves, whose LDS starts at lds, by the same waves
  __device__ __forceinline__ static void activate(const DecodeArgs& a, const Choice& c, int i, int f0, int kw, int wk,
                                                  const unsigned char* lds) {
    const int row0 = c.row0[i], cnt = c.row0[i + 1] - row0, F = a.F;
    const int ln = threadIdx.x & 63;
    for (int o = wk; o < (cnt > 16 ? 16 : 8); o += kw) {
      const int q = o & 3, cb = (o >> 2) & 1, r = (o >> 3) * 16 + (ln & 15), f = f0 + cb * 16 + (ln >> 4) * 4 + q;
      if (r < cnt && f < F) {
        float g = 0.f, u = 0.f;
        auto add = [&](int w) {
          const float* red = reinterpret_cast<const float*>(lds + w * WAVE_LDS);
          g += red[(((o >> 3) * 4 + cb) * 4 + q) * 64 + ln];
          u += red[(((o >> 3) * 4 + 2 + cb) * 4 + q) * 64 + ln];
        };
        if (!ANY_KW || kw == NW) {
#pragma unroll
          for (int w = 0; w < NW; ++w) add(w);
        } else {
          for (int w = 0; w < kw; ++w) add(w);
        }
        const float h = silu(g) * u;
        // the two parts of 32 elements side by side: a 128-byte line per row and fragment load
        bf16_t* to = static_cast<bf16_t*>(a.h) + (int64_t)(row0 + r) * w4_pitch(F) * 2 + w4_place2(f);
        to[0] = (bf16_t)h;
        to[32] = (bf16_t)bf16_rest(h);
      }
    }
  }

  __device__ __forceinline__ static void run(const DecodeArgs& a, const Choice& c, unsigned char* smem) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nft = (a.F + COLS - 1) / COLS, total = __builtin_amdgcn_readfirstlane(c.n) * nft;
    const int ns = (a.H + WS::STEP - 1) / WS::STEP;
    int lw = LW;  // log2 of the waves of a tile
    if (ANY_KW)
      while (lw > 0 && narrow(ns, total, gridDim.x, lw)) --lw;
    const int kw = 1 << lw, wk = wave & (kw - 1), tiles = NW >> lw;
    unsigned char* lds = smem + wave * WAVE_LDS;
    for (int t0 = blockIdx.x * tiles; t0 < total; t0 += gridDim.x * tiles) {
      const int t = t0 + (wave >> lw), i = min(t, total - 1) / nft, f0 = (t - i * nft) * COLS;
      const int n = t < total ? __builtin_amdgcn_readfirstlane(c.row0[i + 1] - c.row0[i]) : 0;
      if (n > 16) multiply<16, 2>(a, c, i, f0, kw, wk, lds);
      else if (n > 4) multiply<16, 1>(a, c, i, f0, kw, wk, lds);
      else if (n > 0) multiply<4, 1>(a, c, i, f0, kw, wk, lds);
      if (kw > 1) __syncthreads();  // one wave's LDS accesses are in order by themselves
      if (n > 0) activate(a, c, i, f0, kw, wk, lds - wk * WAVE_LDS);
      if (kw > 1) __syncthreads();
    }
  }
};

template <typename G>
__global__ __launch_bounds__(512, 4) void decode_gate_up_kernel(DecodeArgs a) {
  constexpr int BYTES = G::NW * G::WAVE_LDS;
  __shared__ Choice c;
  __shared__ __attribute__((aligned(16))) unsigned char
      smem[BYTES > (int)sizeof(ChoiceScratch) ? BYTES : (int)sizeof(ChoiceScratch)];
  choose(a, c, *reinterpret_cast<ChoiceScratch*>(smem), blockIdx.x == 0);  // done with its scratch before the first tile
  __syncthreads();
  G::run(a, c, smem);
}

// ------------------------------------------------------------------------------------------------
// down and combine
// ------------------------------------------------------------------------------------------------
// A tile is 16 columns of y (32 with 4-bit weights) for every token, over all chosen experts. The units (expert, K
// step), expert by expert, are cut into runs, one per wave. Where a run passes from an expert to the next, the wave
// multiplies its sums by the rows' routing weights and adds them to its tokens' sums in LDS; the waves' sums are added
// in wave order. For bf16 layers h has two bf16 parts, hi and lo, so it keeps 16 significant bits: a matrix step's 16
// columns are the hi parts of eight rows and their lo parts, which are added at the end. f32 layers have 16 rows per
// step. The wider 4-bit tiles are half as many, so they take sixteen waves instead of eight.
template <typename T, bool W4>
struct Down {
  static constexpr int NW = W4 ? 16 : 8, NTH = NW * 64;
  static constexpr int CB = W4 ? 2 : 1;                // blocks of 16 columns
  static constexpr int COLS = CB * 16;
  using RS = RowStep<T, 1>;
  using WS = W4Step<CB>;
  static constexpr int STEP = W4 ? WS::STEP : RS::STEP;
  static constexpr int STAGE = W4 ? WS::LDS_BYTES : RS::LDS_BYTES;
  static constexpr int SUMS = MOE_DECODE_MAX_TOKENS * COLS * 4;
  static constexpr int WAVE_LDS = STAGE + SUMS;

  static constexpr int rows(int cw) { return sizeof(T) == 2 ? cw / 2 : cw; }  // rows in cw columns of a matrix step

  // K steps [s_begin, s_end) of one expert for NB blocks of CW columns of its rows from row r0 on (CW 4: 4-bit only)
  template <int NB, int CW>
  __device__ __forceinline__ static void run(const DecodeArgs& a, const Choice& c, int i, int r0, int s_begin, int s_end,
                                             int n0, unsigned char* lds, float* sums) {
    constexpr int PF = W4 ? (NB > 1 ? 1 : CW == 16 ? 3 : 4) : (NB > 1 ? 2 : 4);  // steps of loads in flight
    constexpr int RPB = rows(CW), XV = W4 ? CW / 4 : RS::XV;
    const int lane = threadIdx.x & 63;
    const int K = a.F, H = a.H;
    const int64_t l = __builtin_amdgcn_readfirstlane(c.expert[i]);
    const int row0 = __builtin_amdgcn_readfirstlane(c.row0[i]) + r0;
    const int cnt = __builtin_amdgcn_readfirstlane(c.row0[i + 1]) - row0;
    // elements of a row of h, and from its first to its second part
    const int pitch = W4 ? w4_pitch(K) * 2 : K;
    const int64_t part = W4 ? 32 : (int64_t)a.T * a.k * K;
    const __amdgpu_buffer_rsrc_t hr = __builtin_amdgcn_make_buffer_rsrc(
        (char*)a.h + (int64_t)row0 * pitch * (int)sizeof(T), (short)0,
        (int)((sizeof(T) == 2 && !W4 ? part : 0) + (int64_t)cnt * pitch) * (int)sizeof(T), 0x00020000);
    int cols[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = (lane & 15) % CW, r = nb * RPB + col % RPB;
      cols[nb] = r < cnt ? (r * pitch + (col >= RPB ? (int)part : 0)) * (int)sizeof(T) : -1;
    }
    f32x4 acc[CB][NB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[cb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 rx[PF][NB][XV];
    if constexpr (W4) {
      const int ks = (K + W4_STILE_K - 1) / W4_STILE_K;
      WS ws;
#pragma unroll
      for (int b = 0; b < CB; ++b) ws.block(b, a.w_dn, a.s_dn, (l * H + n0) / 16 + b, K);
      u32x4 rw[PF][CB];
      auto load = [&](int st, int u) {
        const int s = min(st, s_end - 1);
        ws.load(rw[u], s, lane);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) WS::template load_col<2, CW>(rx[u][nb], hr, cols[nb], s, K, lane);
      };
      for (int s0 = s_begin; s0 < s_end;) {
        const int t0 = s0 >> 2, stop = min(s_end, (t0 + WS::CHUNK) * 4);
        u32x4 sv[CB];
        ws.load_scales(sv, t0, ks, lane);
#pragma unroll
        for (int u = 0; u < PF; ++u) load(s0 + u, u);
        WS::store_scales(sv, lds, lane);
        auto use = [&](int st, int u) {
          float sc[CB];
#pragma unroll
          for (int b = 0; b < CB; ++b) sc[b] = WS::scale(lds, b, t0, st, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
              const u32x4 f[1] = {w4_to_bf16(rw[u][cb][j], sc[cb])};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const u32x4 b[1] = {WS::template col<CW>(rx[u][nb], j)};
                Op16::step(acc[cb][nb], f, b);
              }
            }
          }
        };
        pipeline<PF, 1>(s0, stop, use, load);
        s0 = stop;
      }
    } else {
      const T* rows[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        rows[q] = static_cast<const T*>(a.w_dn) + (l * H + min(n0 + q * 8 + (lane >> 3), H - 1)) * K;
      typename RS::Regs rw[PF];
      auto load = [&](int st, int u) {
        const int s = min(st, s_end - 1);
        RS::load(rw[u], rows, s, K, lane);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) RS::load_col(rx[u][nb], hr, cols[nb], s, K, lane);
      };
#pragma unroll
      for (int u = 0; u < PF; ++u) load(s_begin + u, u);
      auto use = [&](int st, int u) {
        RS::stage(rw[u], lds, st, K, lane);
#pragma unroll
        for (int kk = 0; kk < RS::KST; ++kk) {
          u32x4 f[RS::VPF];
          RS::frag(lds, 0, kk, lane, f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            u32x4 b[RS::VPF];
#pragma unroll
            for (int q = 0; q < RS::VPF; ++q) b[q] = rx[u][nb][kk * RS::VPF + q];
            DecOp<T>::step(acc[0][nb], f, b);
          }
        }
      };
      pipeline<PF, 1>(s_begin, s_end, use, load);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            // row_ror: lane c adds the other part, c + RPB
            acc[cb][nb][q] = join_parts(acc[cb][nb][q], dpp_f32<0x120 + 16 - RPB>(acc[cb][nb][q]));
      }
      const int col = lane & 15, r = nb * RPB + col;
      if (col < RPB && r < cnt) {
        const float w = c.w[row0 + r];
        float* y = sums + c.token[row0 + r] * COLS + (lane >> 4) * 4;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int q = 0; q < 4; ++q) y[cb * 16 + q] = fmaf(w, acc[cb][nb][q], y[cb * 16 + q]);
      }
    }
  }

  // part: which of the a.split equal parts of the units
  __device__ __forceinline__ static void tile(const DecodeArgs& a, const Choice& c, int n0, int part,
                                              unsigned char* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ns = (a.F + STEP - 1) / STEP, units = c.n * ns;
    const int runs = NW * a.split, run_id = part * NW + wave;
    const int per = (units + runs - 1) / runs;
    const int u_end = min(units, (run_id + 1) * per);
    unsigned char* lds = smem + wave * WAVE_LDS;
    float* sums = reinterpret_cast<float*>(lds + STAGE);
    for (int o = lane; o < a.T * COLS; o += 64) sums[o] = 0.f;
    for (int u = min(units, run_id * per); u < u_end;) {
      const int i = __builtin_amdgcn_readfirstlane(u / ns), s = u - i * ns;
      const int n = min(ns - s, u_end - u);
      const int cnt = c.row0[i + 1] - c.row0[i];
      constexpr int RPB = rows(16);
      // more than two blocks: two at a time, the weights again from L2 (one expert's run is a few KB)
      if (W4 && cnt <= rows(4)) run<1, W4 ? 4 : 16>(a, c, i, 0, s, s + n, n0, lds, sums);
      else if (cnt <= RPB) run<1, 16>(a, c, i, 0, s, s + n, n0, lds, sums);
      else
        for (int r0 = 0; r0 < cnt; r0 += 2 * RPB) run<2, 16>(a, c, i, r0, s, s + n, n0, lds, sums);
      u += n;
    }
    __syncthreads();
    for (int o = tid; o < a.T * COLS; o += NTH) {
      const int r = o % COLS, t = o / COLS;
      if (n0 + r < a.H) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += reinterpret_cast<const float*>(smem + w * WAVE_LDS + STAGE)[o];
        if (a.split > 1) a.partial[((int64_t)part * a.T + t) * a.H + n0 + r] = v;
        else static_cast<T*>(a.y)[(int64_t)t * a.H + n0 + r] = from_f32<T>(v);
      }
    }
    __syncthreads();
  }
};

template <typename T, bool W4>
__global__ __launch_bounds__((Down<T, W4>::NTH), 4) void decode_down_kernel(DecodeArgs a) {
  using D = Down<T, W4>;
  __shared__ Choice c;
  __shared__ __attribute__((aligned(16))) unsigned char smem[D::NW * D::WAVE_LDS];
  for (int x = threadIdx.x; x < (int)(sizeof(Choice) / 4); x += D::NTH)
    reinterpret_cast<int*>(&c)[x] = reinterpret_cast<const int*>(a.choice)[x];
  __syncthreads();
  const int total = (a.H + D::COLS - 1) / D::COLS * a.split;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x)
    D::tile(a, c, tile / a.split * D::COLS, tile % a.split, smem);
}

// y of a split down kernel: the parts' sums, added in their order
template <typename T>
__global__ __launch_bounds__(256) void decode_sum_kernel(DecodeArgs a) {
  const int64_t n = (int64_t)a.T * a.H, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.split; ++p) v += *reinterpret_cast<const f32x4*>(a.partial + p * n + i);
#pragma unroll
  for (int q = 0; q < 4; ++q) static_cast<T*>(a.y)[i + q] = from_f32<T>(v[q]);
}

// Parts of the down kernel's units, for an H whose tiles leave half of the CUs idle: as many as give every CU its
// workgroups, with eight steps per wave at least, since adding the parts takes one more launch. Whole layers (us,
// without and with; T tokens, E experts, k of them each):
//   f32  T 13, E 37, k 4, H 968, F 4992      477   323
//   bf16 T 32, E 64, k 8, H 1024, F 1024     127    92
//   bf16 T  8, E  8, k 2, H 2048, F 8192     149   142
//   bf16 T  4, E 16, k 2, H 3584, F 4096     108   115   (224 tiles: not split)
//   w4   T 16, E 64, k 4, H 1024, F 4096     115    67
//   w4   T 16, E 32, k 4, H 2880, F 2880     104    89
//   w4   T  1, E 128, k 8, H 2048, F 768    17.3  17.3   (too few steps: not split)
constexpr int kDownSplit = 8;         // parts at most
constexpr int kDownSplitMaxH = 4096;  // no wider: the workspace has no room for the parts there
int down_split(const DecodeArgs& a, int cols, int step, int nw, int num_cus) {
  const int tiles = ceil_div_host(a.H, cols);
  if (a.H > kDownSplitMaxH || tiles > num_cus / 2) return 1;
  const int64_t units = (int64_t)std::min(a.T * a.k, a.El) * ceil_div_host(a.F, step);
  const int64_t s = std::min<int64_t>({kDownSplit, 16 / nw * num_cus / tiles, units / nw / 8});
  return s < 2 ? 1 : (int)s;
}

template <typename T>
void launch_route_rows(const T* x, const float* w, const float* bias, int64_t bias_stride, int T_, int H, int E,
                       float* logits, bf16_t* placed, hipStream_t stream) {
  auto go = [&](auto tb, auto eb) {
    constexpr int TB = decltype(tb)::value, EB = decltype(eb)::value;
    decode_route_kernel<T, TB, EB><<<dim3(ceil_div_host(E, EB), ceil_div_host(T_, TB)), 256, 0, stream>>>(
        x, w, bias, bias_stride, T_, H, E, logits, placed);
  };
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C4 = std::integral_constant<int, 4>;
  // Four tokens and as many experts as leave a few workgroups per CU: a workgroup's loads of a step are all in flight
  // together. 384 experts, H 7168 (us): 32 tokens 4 x 4 9.4, 8 x 2 9.8, 8 x 4 10.6, 8 x 1 11.5; 16 tokens 4 x 2 6.7,
  // 8 x 1 7.5, 8 x 4 9.0
  if (T_ == 1) go(C1{}, C1{});
  else if (T_ == 2) go(C2{}, C1{});
  else if (T_ <= 4 || E < 128) go(C4{}, C1{});
  else if (T_ <= 16 || E < 256) go(C4{}, C2{});
  else go(C4{}, C4{});
}

template <typename T, bool W4>
void launch_experts(DecodeArgs a, int num_cus, hipStream_t stream) {
  using G = std::conditional_t<W4, GateUpW4<false>, GateUp<T, 1>>;
  using D = Down<T, W4>;
  const int64_t gu = (int64_t)std::min(a.T * a.k, a.El) * ceil_div_host(a.F, G::COLS);
  const int grid = (int)std::min<int64_t>(gu, 2 * num_cus);
  if constexpr (W4) {
    if (G::narrow(ceil_div_host(a.H, W4_TILE_K), gu, grid, G::LW))
      decode_gate_up_kernel<GateUpW4<true>><<<grid, G::NTH, 0, stream>>>(a);
    else
      decode_gate_up_kernel<G><<<grid, G::NTH, 0, stream>>>(a);
  } else {
    if (a.T <= 16) decode_gate_up_kernel<GateUp<T, 1>><<<grid, GateUp<T, 1>::NTH, 0, stream>>>(a);
    else decode_gate_up_kernel<GateUp<T, 2>><<<grid, GateUp<T, 2>::NTH, 0, stream>>>(a);
  }
  a.split = down_split(a, D::COLS, D::STEP, D::NW, num_cus);
  const int tiles = ceil_div_host(a.H, D::COLS) * a.split;
  decode_down_kernel<T, W4><<<std::min(tiles, 16 / D::NW * num_cus), D::NTH, 0, stream>>>(a);
  if (a.split > 1)
    decode_sum_kernel<T><<<(unsigned)ceil_div_host64((int64_t)a.T * a.H, 1024), 256, 0, stream>>>(a);
}

}  // namespace

size_t decode_workspace_bytes(int T, int H, int k, int F) {
  return align256(sizeof(Choice)) + align256((size_t)T * k * (size_t)w4_pitch(F) * 4) +
         align256((size_t)T * (size_t)w4_pitch(H) * 2) +
         (H <= kDownSplitMaxH ? (size_t)kDownSplit * T * (size_t)H * 4 : 0);
}

hipError_t launch_layer_decode(const DecodeCall& d, int num_cus, hipStream_t stream) {
  char* ws = static_cast<char*>(d.workspace);
  DecodeArgs a{};
  a.choice = reinterpret_cast<Choice*>(ws);
  ws += align256(sizeof(Choice));
  a.h = ws;
  ws += align256((size_t)d.T * d.k * (size_t)w4_pitch(d.F) * 4);
  bf16_t* placed = d.s_gu ? reinterpret_cast<bf16_t*>(ws) : nullptr;
  a.partial = reinterpret_cast<float*>(ws + align256((size_t)d.T * (size_t)w4_pitch(d.H) * 2));
  if (d.bf16)
    launch_route_rows(static_cast<const bf16_t*>(d.x), d.w_router, d.bias, d.bias_stride, d.T, d.H, d.E, d.logits,
                      placed, stream);
  else
    launch_route_rows(static_cast<const float*>(d.x), d.w_router, d.bias, d.bias_stride, d.T, d.H, d.E, d.logits,
                      nullptr, stream);
  a.x = placed ? placed : d.x;
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
  if (!d.bf16) launch_experts<float, false>(a, num_cus, stream);
  else if (d.s_gu) launch_experts<bf16_t, true>(a, num_cus, stream);
  else launch_experts<bf16_t, false>(a, num_cus, stream);
  return hipGetLastError();
}

}  // namespace moe
