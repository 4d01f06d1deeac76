// The balance loss of a router, its per-expert counts and its gradient (moe_balance_loss).
//
// A sequence s has n counted tokens; expert e has count[s, e] of their choices, f = count / (k n). With p = softmax of a
// token's logits the sequence's loss is E / n sum_t sum_e f p, and, as f does not depend on the logits, a token's gradient is
// E / n p (f - sum f p). The loss is linear in the tokens' dot products sum f p, which the gradient needs too: nothing but
// the counts has to be known before the one pass over the logits. f enters less its smallest value over the experts, which the
// gradient does not depend on: where the choices are nearly even the difference, taken of the counts, then keeps its digits, and
// it is 0 where they are even (k = E); no term is larger than without.
//
//   balance_count   counts of each sequence's ids, in `splits` parts that need no clearing and no float atomics
//   balance_rows    one pass over the logits: a group of lanes per token (softmax, dot product, gradient), a double partial of
//                   the loss per workgroup; the workgroup that finishes last adds the partials in their order
// Bound: 8 bytes per logit (read, gradient written) and the ids, at HBM rates for large batches; two launches for small ones.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "tiles.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int NTH = 1024, NW = NTH / 64;

struct BalanceArgs {
  const float* logits;
  const int* ids;
  const int* seq_offset;  // [S + 1], or nullptr: one sequence of all tokens
  const uint8_t* mask;    // [T], or nullptr
  int T, E, k, S, splits;
  float weight;
  int* part;        // [S, splits, E + 1]: counts, then counted tokens
  double* partial;  // [workgroups of balance_rows]
  int* ticket;
  float* loss;
  int* count;       // [S, E]
  float* d_logits;  // [T, E] or nullptr
};

// Tokens [begin, end) of sequence s, within [0, T) whatever the offsets hold.
__device__ __forceinline__ void seq_range(const BalanceArgs& a, int s, int& begin, int& end) {
  begin = a.seq_offset ? min(max(a.seq_offset[s], 0), a.T) : 0;
  end = a.seq_offset ? min(max(a.seq_offset[s + 1], begin), a.T) : a.T;
}

// Workgroup (split, s): the ids of one part of sequence s into LDS counters, and from there to the part's own place.
__global__ __launch_bounds__(NTH) void balance_count_kernel(BalanceArgs a) {
  __shared__ int s_count[MOE_MAX_EXPERTS + 1];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *a.ticket = 0;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    for (int e = tid; e <= a.E; e += NTH) s_count[e] = 0;
    __syncthreads();
    int begin, end;
    seq_range(a, s, begin, end);
    const int64_t per = ((int64_t)(end - begin) + a.splits - 1) / a.splits;
    const int64_t t0 = begin + blockIdx.x * per, t1 = min((int64_t)end, t0 + per);
    int tokens = 0;
    for (int64_t t = t0 + tid; t < t1; t += NTH) tokens += !a.mask || a.mask[t] != 0;
    for (int64_t i0 = t0 * a.k + tid; i0 < t1 * a.k; i0 += 8 * NTH) {  // eight loads in flight
      int e[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int64_t i = i0 + q * NTH;
        const bool in = i < t1 * a.k;
        e[q] = in ? a.ids[i] : -1;
        if (a.mask && in && a.mask[(unsigned)i / (unsigned)a.k] == 0) e[q] = -1;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (e[q] >= 0 && e[q] < a.E) atomicAdd(&s_count[e[q]], 1);
    }
    if (tokens) atomicAdd(&s_count[a.E], tokens);
    __syncthreads();
    int* out = a.part + ((int64_t)s * a.splits + blockIdx.x) * (a.E + 1);
    for (int e = tid; e <= a.E; e += NTH) out[e] = s_count[e];
    __syncthreads();
  }
}

// Sum and maximum over a group of 4, 16 or 64 lanes, in every lane, in a fixed order (DPP within the 16 lanes of a row)
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G == 64) return wave_sum(v);
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  if constexpr (G == 16) {
    v += dpp_f32<0x141>(v);
    v += dpp_f32<0x140>(v);
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (G == 64) return wave_max(v);
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  if constexpr (G == 16) {
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
  }
  return v;
}

template <int G>
__device__ __forceinline__ int group_max_i32(int v) {
  if constexpr (G == 64) return wave_max_i32(v);
  v = max(v, dpp_i32<0xB1>(v));
  v = max(v, dpp_i32<0x4E>(v));
  if constexpr (G == 16) {
    v = max(v, dpp_i32<0x141>(v));
    v = max(v, dpp_i32<0x140>(v));
  }
  return v;
}

// Entry e of sequence s over its parts, whose loads go out together (one after another they are 16 round trips: 7 us)
constexpr int kMaxSplits = 16;
__device__ __forceinline__ int part_sum(const BalanceArgs& a, int64_t s, int64_t e) {
  int v[kMaxSplits], c = 0;
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) v[i] = i < a.splits ? a.part[(s * a.splits + i) * (a.E + 1) + e] : 0;
#pragma unroll
  for (int i = 0; i < kMaxSplits; ++i) c += v[i];
  return c;
}

// G lanes per token, NV vectors of VW logits per lane: lane i of the group holds logits (i + j G) VW .. of j < NV.
// A workgroup takes `tokens` consecutive tokens; where they belong to several sequences it goes through these in turn, with
// the sequence's counts in LDS. A group loads U tokens at once: a large batch is one such round, and its loads are what it waits
// for (one token after another: 30 us for 16384 x 256, 16 with four at once).
// MANY: more than kFewSeqs sequences, whose tokens would be few at a time: a group finds its token's sequence and reads its
// counts itself, which have to be in one part. Kernel times (us) one sequence after another, and so:
//   tokens x experts, sequences   301 x 24, 9   301 x 24, 16   4000 x 24, 9   4000 x 256, 9   4000 x 256, 16   16384 x 256, 16
//                                    13.7  6.3     17.2   6.5     11.1   8.7      15.2  10.5       15.6  10.8        20.2   19.9
// Fewer sequences are counted in parts where the batch is large (16 / S of them from 4096 / S tokens on), hence the border.
// Batches of under 512 tokens have one part: below it, they would take 6.0 us so at two sequences of 24 experts instead of 10.4,
// 6.2 instead of 10.8 at five, and 8.0 instead of 19.5 at eight of 256.
constexpr int kFewSeqs = 8;
template <int G, int VW, int NV, bool MANY>
__global__ __launch_bounds__(NTH) void balance_rows_kernel(BalanceArgs a, int tokens) {
  constexpr int TPP = NTH / G, U = MANY ? 1 : NV > 2 ? 2 : 4;  // tokens per pass, passes at once
  __shared__ int s_count[MOE_MAX_EXPERTS];
  __shared__ double s_sum[NW];
  __shared__ int s_n, s_used, s_last;
  const int tid = threadIdx.x, gl = tid % G;
  const int t_begin = blockIdx.x * tokens, t_end = min(a.T, t_begin + tokens);
  // sequences with counted tokens
  if (tid == 0) s_used = 0;
  __syncthreads();
  if (a.S > 1) {
    int used = 0;
    for (int s = tid; s < a.S; s += NTH) used += part_sum(a, s, a.E) > 0;
    if (used) atomicAdd(&s_used, used);
  }
  // This lane's f less the smallest f, which it returns, of a sequence of n tokens (0 if there are none) from its counts
  auto shares = [&](auto&& count, int n, float (&f)[NV][VW]) {
    const float unit = n > 0 ? 1.f / ((float)a.k * (float)n) : 0.f;
    int c[NV][VW], least = INT32_MAX;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VW; ++q) {
        const int e = (gl + j * G) * VW + q;
        c[j][q] = n > 0 && e < a.E ? count(e) : 0;
        least = e < a.E ? min(least, c[j][q]) : least;
      }
    least = -group_max_i32<G>(-least);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VW; ++q) f[j][q] = (gl + j * G) * VW + q < a.E ? (float)(c[j][q] - least) * unit : 0.f;
    return (float)least * unit;
  };
  // softmax, loss and gradient of token t, whose logits are x; f, least and factor are its sequence's
  double sum = 0.0;
  auto token = [&](int t, bool write, bool live, float (&x)[NV][VW], const float (&f)[NV][VW], float least, float factor) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VW; ++q) m = fmaxf(m, x[j][q]);
    m = group_max<G>(m);
    const float base = m == -INFINITY ? 0.f : m;  // every logit -inf: p is 0 and the token adds nothing
    float z = 0.f, d = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VW; ++q) {
        x[j][q] = expf(x[j][q] - base);
        z += x[j][q];
        d = fmaf(x[j][q], f[j][q], d);
      }
    z = group_sum<G>(z);
    d = group_sum<G>(d);
    const float iz = z > 0.f ? 1.f / z : z == 0.f ? 0.f : z;  // NaN stays NaN
    const float dot = d * iz;
    if (gl == 0 && live) sum += (double)(factor * (dot + (z > 0.f ? least : z)));
    if (a.d_logits && write) {
      float* out = a.d_logits + (int64_t)t * a.E;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = (gl + j * G) * VW;
        if (e < a.E) {
          float o[VW];
#pragma unroll
          for (int q = 0; q < VW; ++q) o[q] = live ? factor * (x[j][q] * iz) * (f[j][q] - dot) : 0.f;
          if constexpr (VW == 4) st16_nt(out + e, pack(o));
          else out[e] = o[0];
        }
      }
    }
  };
  auto load = [&](int t, bool live, float (&x)[NV][VW]) {
    const float* row = a.logits + (int64_t)t * a.E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (gl + j * G) * VW;
      if constexpr (VW == 4) {
        u32x4 v{0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
        if (live && e < a.E) v = ld16_nt(row + e);
        unpack(v, x[j]);
      } else {
        x[j][0] = live && e < a.E ? row[e] : -INFINITY;
      }
    }
  };
  if constexpr (MANY) {
    __syncthreads();  // s_used
    for (int t = t_begin + tid / G; t < t_end; t += TPP) {
      int s = 0;  // the last sequence that begins at or before the token
      for (int hi = a.S; hi - s > 1;) {
        const int mid = (s + hi) >> 1;
        if (a.seq_offset[mid] <= t) s = mid;
        else hi = mid;
      }
      int begin, end;
      seq_range(a, s, begin, end);
      const int n = t >= begin && t < end ? a.part[(int64_t)s * (a.E + 1) + a.E] : 0;
      const bool live = n > 0 && (!a.mask || a.mask[t] != 0);
      float x[NV][VW], f[NV][VW];
      load(t, live, x);
      const float least = shares([&](int e) { return a.part[(int64_t)s * (a.E + 1) + e]; }, n, f);
      token(t, true, live, x, f, least, n > 0 ? a.weight * (float)a.E / ((float)n * (float)s_used) : 0.f);
    }
  } else {
    // the sequence of the first token: the last one that begins at or before it
    int s = 0;
    for (int hi = a.S; hi - s > 1;) {
      const int mid = (s + hi) >> 1;
      if (a.seq_offset[mid] <= t_begin) s = mid;
      else hi = mid;
    }
    int t0 = t_begin;
    while (t0 < t_end) {
      int begin = 0, end = 0;
      if (s < a.S) seq_range(a, s, begin, end);
      // tokens from t0 on that share a sequence, or share having none
      int t1 = t_end;
      bool in = false;
      if (s < a.S) {
        in = t0 >= begin && t0 < end;
        t1 = in ? min(t_end, end) : t0 < begin ? min(t_end, begin) : t0;
      }
      if (t1 > t0) {
        __syncthreads();  // s_count has been read
        if (in) {
          for (int e = tid; e <= a.E; e += NTH) {
            const int c = part_sum(a, s, e);
            if (e < a.E) s_count[e] = c;
            else s_n = c;
          }
        }
        __syncthreads();
        const int n = in ? s_n : 0;
        const float factor = n > 0 ? a.weight * (float)a.E / ((float)n * (float)(a.S > 1 ? s_used : 1)) : 0.f;
        float f[NV][VW];
        const float least = shares([&](int e) { return s_count[e]; }, n, f);
        for (int tu = t0 + tid / G; tu < t1; tu += TPP * U) {
          float x[U][NV][VW];
          bool live[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int t = tu + u * TPP;
            live[u] = n > 0 && t < t1 && (!a.mask || a.mask[t] != 0);
            load(t, live[u], x[u]);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) token(tu + u * TPP, tu + u * TPP < t1, live[u], x[u], f, least, factor);
        }
        t0 = t1;
      }
      if (s < a.S && t0 >= end) ++s;
    }
  }
  // counts of the whole batch, a slice per workgroup
  for (int64_t i = (int64_t)blockIdx.x * NTH + tid; i < (int64_t)a.S * a.E; i += (int64_t)gridDim.x * NTH) {
    const int64_t sq = i / a.E;
    a.count[i] = part_sum(a, sq, i - sq * a.E);
  }
  // the workgroup's partial, at agent scope; the last workgroup to have stored its own adds them all
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    double v = 0.0;
    for (int w = 0; w < NW; ++w) v += s_sum[w];
    __hip_atomic_store(&a.partial[blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // an agent-scope store writes through to where every XCD reads it: its acknowledgement is all the order it needs (the
    // release and acquire that the memory model asks for beside it are for plain accesses, which the L2s may hold: with them
    // 17.5 us instead of 15.4 for 16384 x 256, as the write-back flushes the gradients as well)
    wait_loads<0>();
    s_last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  double v = 0.0;
  for (int i = tid; i < (int)gridDim.x; i += NTH)
    v += __hip_atomic_load(&a.partial[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((tid & 63) == 0) s_sum[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    v = 0.0;
    for (int w = 0; w < NW; ++w) v += s_sum[w];
    *a.loss = (float)v;
  }
}

// Tokens per workgroup of balance_rows: a workgroup for every CU. More of them would queue for the one ticket.
constexpr int kMaxGroups = 256;
int rows_per_group(int T) { return std::max(16, ceil_div_host(T, kMaxGroups)); }
static_assert(kMaxSplits / (kFewSeqs + 1) <= 1, "many sequences are not counted in parts");
int count_splits(int T, int S) { return std::max(1, std::min(kMaxSplits / S, T / 256)); }

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  return 256 + align256((size_t)std::max(1, ceil_div_host(T, rows_per_group(T))) * sizeof(double)) +
         align256((size_t)S * count_splits(T, S) * (size_t)(E + 1) * sizeof(int));
}

hipError_t launch_balance(const float* logits, const int* ids, const int* seq_offset, const uint8_t* mask, int T, int E,
                          int k, int S, float weight, float* loss, int* count, float* d_logits, void* workspace,
                          hipStream_t stream) {
  const int tokens = rows_per_group(T), groups = std::max(1, ceil_div_host(T, tokens));
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.seq_offset = S == 1 && !seq_offset ? nullptr : seq_offset;
  a.mask = mask;
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.splits = count_splits(T, S);
  a.weight = weight;
  a.ticket = reinterpret_cast<int*>(ws);
  a.partial = reinterpret_cast<double*>(ws + 256);
  a.part = reinterpret_cast<int*>(ws + 256 + align256((size_t)groups * sizeof(double)));
  a.loss = loss;
  a.count = count;
  a.d_logits = d_logits;
  balance_count_kernel<<<dim3(a.splits, std::min(S, 65535)), NTH, 0, stream>>>(a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
#define MOE_BALANCE(G, VW, NV)                                                             \
  do {                                                                                    \
    if (S > kFewSeqs) balance_rows_kernel<G, VW, NV, true><<<groups, NTH, 0, stream>>>(a, tokens); \
    else balance_rows_kernel<G, VW, NV, false><<<groups, NTH, 0, stream>>>(a, tokens);     \
  } while (0)
  if (E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0 && (reinterpret_cast<uintptr_t>(d_logits) & 15) == 0) {
    if (E <= 16) MOE_BALANCE(4, 4, 1);
    else if (E <= 64) MOE_BALANCE(16, 4, 1);
    else if (E <= 256) MOE_BALANCE(64, 4, 1);
    else MOE_BALANCE(64, 4, 2);
  } else {
    if (E <= 16) MOE_BALANCE(16, 1, 1);
    else if (E <= 64) MOE_BALANCE(64, 1, 1);
    else if (E <= 128) MOE_BALANCE(64, 1, 2);
    else MOE_BALANCE(64, 1, 8);
  }
#undef MOE_BALANCE
  return hipGetLastError();
}

}  // namespace moe
