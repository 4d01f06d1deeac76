// Expert SwiGLU MLP on dispatched int8 rows with int8 expert weights (moe_expert_mlp_i8).
//
//   gate/up   g = s_row s_ch (sum_k q_x q_w), u alike: the products are int8, their sums int32 and exact; h = silu(g) u
//             in float32, and the largest |h| of each row of a tile
//   h rows    a row's maximum is that of its tiles; h to int8 codes with the row's scale
//   down      out = s_h s_ch (sum_f q_h q_w), rounded once to bf16
// The plan (rows grouped by local expert, mlp.hip) is moe_expert_mlp's. h stays float32 until its codes: any shorter form
// would move codes over their borders, which a row's maximum, known only after the whole pass, decides.
//
//   i8_gemm_kernel  rows and weight rows go to LDS directly, in stages of 128 k (128 bytes of a row: whole cache lines), NS
//                   stages in flight; 32- and 64-row tiles stream the weights of experts with few rows and are bound by their
//                   bytes (48 experts of 7168 x 2048, 128 tokens: gate/up 213 us, 6.6 TB/s, down 113, 6.2 TB/s), 128- and
//                   256-row ones by the matrix units and the power that they draw (32 experts of 7168 x 2048, 1024 rows each:
//                   gate/up 975-990 us, down 535-560, 1.9 PFLOP/s at 1.8 GHz).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "i8.h"
#include "kernels.h"
#include "mfma.h"
#include "tiles.h"
#include "topk.h"

namespace moe {

namespace {

struct I8Args {
  const int8_t* A;       // rows [., K]: the send rows, or the codes of h in plan order
  const int* a_perm;     // source row of a plan row, or nullptr (A in plan order)
  const float* a_scale;  // [rows of A]
  const int8_t* W;       // [El, w_rows, K]
  const float* w_scale;  // [El, w_rows]
  int K, N;              // N: output columns (F or H)
  int w_rows;            // weight rows per expert (2F or H)
  int up;                // weight row of the up half (gate/up only)
  float* h;              // gate/up: [., N] in plan order
  uint32_t* h_top;       // gate/up: [., h_tiles] bits of the largest |h| of a row in each tile of columns
  int h_tiles;
  bf16_t* out;           // down: [., N]
  const int* out_perm;   // down: destination row of a plan row
  // row_start [El + 1]: first plan row of each expert, the last entry all rows. tile_start [El + 1]: first tile of BM rows, or
  // nullptr: each workgroup counts the tiles itself
  const int* row_start;
  const int* tile_start;
  int El;
  // SPLIT: K in `split` parts of split_stages stages each. Gate/up: their int32 sums to partial [split, rows, w_rows]. Down: a
  // thread's sums of a part to partial [tile, split, .., thread], and the workgroup that completes a tile by its count in
  // `ticket` (zeroed by the gate/up kernel) adds them.
  int split, split_stages;
  int* partial;
  int64_t partial_stride;  // gate/up: elements of one part
  int* ticket;
  int* zero;               // gate/up: ints to zero for the down pass
  int zero_n;
};

// g / (1 + e^-g), from 2^t = e^-|g|, which cannot overflow: g / (1 + 2^t) for g >= 0, g 2^t / (1 + 2^t) below. t is a whole number
// n and a rest, taken with what a float leaves of |g| / ln 2, and n goes into exponents: g 2^t is rounded where it is subnormal
// itself, 2^t alone would be lost before (g below -87: a row's codes and scale depend on its values' ratios, however small they
// are). Off by two or three steps: exp2 and the reciprocal are the hardware's, off by one each. The library's expf and division
// cost a tile of the gate/up pass as much as three of its stages.
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299e-8f;  // 1 / ln 2 and what float leaves of it
  const float x = fminf(fabsf(g), 256.f);  // e^-256 is 0 beside and times any float32
  const float t = x * -kLog2e, n = rintf(t);
  const float rest = (t - n) + fmaf(x, -kLog2eLow, fmaf(x, -kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(rest);
  const float top = g < 0.f ? ldexpf(g * e, (int)n) : g;
  return top * __builtin_amdgcn_rcpf(1.0f + ldexpf(e, (int)n));
}

// A stage's rows: 128 bytes each, 16-byte chunk c of row r at c ^ ((r >> 1) & 7), so that a fragment read touches every
// bank once.
__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }

// BM rows x BN weight rows per tile (gate/up: the gate and the up rows of BN / 2 columns), WM x WN waves.
// PP: eight waves in two groups, one of each on every SIMD, that run the same sequence (read half a stage of fragments,
// barrier, multiply them, barrier) one barrier apart: while one group reads and loads the other keeps the matrix units busy.
// Four waves of 128 x 128, reads and loads spread between the products, read a third less LDS and were no faster: gate/up 1025 us
// against 972, down 643 against 557, of which the longer epilogue is most. Nor did it change anything to look up rows and
// scales behind the first loads instead of before them, or to store a lane's neighbouring columns directly.
// SPLIT: K cut over workgroups, where the tiles are few (see i8_plan).
// FEW: a down pass of at most kFewRows rows in all, which takes h itself and makes the codes of its part of K while the first
// weights are on their way, in place of a launch for them (one Mixtral-shaped token 85 -> 75 us with the join in the kernel).
constexpr int kFewRows = 8, kFewStages = 32;
template <typename Op, int BM, int BN, int WM, int WN, int NS, int PER_CU, bool PP, bool GATED, bool SPLIT = false,
          bool FEW = false>
__global__ __launch_bounds__(WM * WN * 64, PER_CU * WM * WN / 4 > 1 ? PER_CU * WM * WN / 4 : 1) void i8_gemm_kernel(
    I8Args a, int a_bytes) {
  static_assert(!PP || (NS == 2 && WM * WN == 8 && !SPLIT), "ping-pong");
  static_assert(!FEW || (SPLIT && !GATED && WM == 1), "a few rows");
  constexpr int S = Op::S, NW = WM * WN, NTH = NW * 64, ROWB = 128, RPI = 8;
  constexpr int SA = FEW ? 0 : BM;                               // rows that a stage loads
  constexpr int A_BYTES = FEW ? kFewStages * kFewRows * ROWB : 0;  // FEW: codes of all stages, before the weights' stages
  constexpr int STAGE = (SA + BN) * ROWB, A_INS = SA / RPI, LPW = (SA + BN) / RPI / NW;
  static_assert((SA + BN) / RPI % NW == 0, "wave loads must split evenly");
  constexpr int OUTC = GATED ? BN / 2 : BN;
  constexpr int WTM = BM / WM, TM = WTM / S, WTN = OUTC / WN, TN = WTN / S;
  constexpr int NACC = GATED ? 2 * TN : TN, KSTEPS = ROWB / Op::KS;
  static_assert(TM >= 1 && TN >= 1, "wave tile too small");
  constexpr int OUT_BYTES = GATED ? 0 : BM * OUTC * 2;
  constexpr int BODY = A_BYTES + NS * STAGE > OUT_BYTES ? A_BYTES + NS * STAGE : OUT_BYTES;
  constexpr int OOB = 0x7ffffff0;
  // the only LDS object (a second one makes the compiler wait for every load in flight before LDS reads): the stages, which
  // the output tile reuses; the tile's row scales and destination rows; the waves' row maxima; the plan's starts
  constexpr int SCALE_OFF = BODY, ROW_OFF = SCALE_OFF + BM * 4, TOP_OFF = ROW_OFF + BM * 4;
  constexpr int PLAN_OFF = TOP_OFF + (GATED ? WN * (S / 16) * BM * 4 : 16);
  __shared__ __attribute__((aligned(1024))) unsigned char smem[PLAN_OFF + 2 * (MOE_MAX_EXPERTS + 1) * 4];
  float* s_scale = reinterpret_cast<float*>(smem + SCALE_OFF);
  int* s_row = reinterpret_cast<int*>(smem + ROW_OFF);
  uint32_t* s_top = reinterpret_cast<uint32_t*>(smem + TOP_OFF);
  int* row_start = reinterpret_cast<int*>(smem + PLAN_OFF);
  int* tile_start = row_start + MOE_MAX_EXPERTS + 1;
  int tid = threadIdx.x, lane = tid & 63;  // made opaque at each tile start (below)
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int fr = lane % S, fq = lane / S;
  const int K = a.K, nk = (K + ROWB - 1) / ROWB;
  if constexpr (GATED)
    for (int i = blockIdx.x * NTH + tid; i < a.zero_n; i += gridDim.x * NTH) a.zero[i] = 0;
  for (int i = tid; i <= a.El; i += NTH) {
    row_start[i] = a.row_start[i];
    if (a.tile_start) tile_start[i] = a.tile_start[i];
  }
  const int n_tiles = (a.N + OUTC - 1) / OUTC;
  __syncthreads();
  if (!a.tile_start) {
    if (wave == 0) {  // an exclusive scan of the experts' tiles, 64 at a time
      int before = 0;
      for (int i0 = 0; i0 < a.El; i0 += 64) {
        const int i = i0 + lane;
        const int n = i < a.El ? (row_start[i + 1] - row_start[i] + BM - 1) / BM : 0;
        int sum = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int up = __shfl_up(sum, off, 64);
          if (lane >= off) sum += up;
        }
        if (i < a.El) tile_start[i] = before + sum - n;
        before += __shfl(sum, 63, 64);
      }
      if (lane == 0) tile_start[a.El] = before;
    }
    __syncthreads();
  }
  const Tiles mine = my_tiles(__builtin_amdgcn_readfirstlane(tile_start[a.El]) * n_tiles * (SPLIT ? a.split : 1));
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.A, (short)0, a_bytes, 0x00020000);
  int l = 0;
  for (int unit = mine.begin; unit < mine.end; unit += mine.step) {
    const int tile = SPLIT ? unit / a.split : unit, sp = SPLIT ? unit - tile * a.split : 0;
    const int s_begin = SPLIT ? sp * a.split_stages : 0, s_end = SPLIT ? min(nk, s_begin + a.split_stages) : nk;
    // per-lane values are computed again in each tile: kept across the tile loop they do not fit the registers next
    // to the accumulators
    asm volatile("" : "+v"(tid), "+v"(lane), "+v"(fr), "+v"(fq));
    // tiles list (expert, N tile, M tile) in expert order and a workgroup's tiles increase: scan on
    while (__builtin_amdgcn_readfirstlane(tile_start[l + 1]) * n_tiles <= tile) ++l;
    const int ts = __builtin_amdgcn_readfirstlane(tile_start[l]);
    const int mt_l = __builtin_amdgcn_readfirstlane(tile_start[l + 1]) - ts;
    const int local = tile - ts * n_tiles;
    const int nt = local / mt_l, mt = local % mt_l;
    const int p0 = __builtin_amdgcn_readfirstlane(row_start[l]) + mt * BM;
    const int m_rows = min(BM, __builtin_amdgcn_readfirstlane(row_start[l + 1]) - p0);
    const int n0 = nt * OUTC;
    const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.W + (int64_t)l * a.w_rows * K), (short)0, a.w_rows * K, 0x00020000);
    const float* w_scale = a.w_scale + (int64_t)l * a.w_rows;

    // this wave's LPW loads of a stage, 8 rows each: the byte offset without k. The source rows are looked up together.
    int voff[LPW];
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
      const int p = p0 + min((wave * LPW + q) * RPI + (lane >> 3), m_rows - 1);
      voff[q] = a.a_perm && wave * LPW + q < A_INS ? a.a_perm[p] : p;
    }
    wait_loads<0>();
    lds_barrier();  // the previous tile has left LDS
    for (int r = tid; r < BM; r += NTH) {
      const int p = p0 + min(r, m_rows - 1);
      if constexpr (!FEW) s_scale[r] = a.a_scale[a.a_perm ? a.a_perm[p] : p];
      s_row[r] = a.out_perm ? a.out_perm[p] : p;
    }
    if constexpr (FEW)
      for (int r = wave; r < BM; r += NW) {  // the rows' maxima, for now
        uint32_t top = 0;
        for (int i = lane; i < a.h_tiles; i += 64) top = max(top, a.h_top[(int64_t)(p0 + min(r, m_rows - 1)) * a.h_tiles + i]);
        top = wave_top(top);
        if (lane == 0) s_scale[r] = __uint_as_float(top);
      }
    int tail = 0;  // bit q: this lane's chunk of load q lies within K in the last stage
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
      const int ins = wave * LPW + q;
      const int r = (ins < A_INS ? ins : ins - A_INS) * RPI + (lane >> 3);
      const int chunk = (lane & 7) ^ swizzle(r);
      tail |= ((nk - 1) * ROWB + chunk * 16 < K ? 1 : 0) << q;
      if (ins < A_INS) {
        voff[q] = r < m_rows ? voff[q] * K + chunk * 16 : OOB;
      } else {
        const int half = GATED ? r / OUTC : 0, col = n0 + (GATED ? r % OUTC : r);
        voff[q] = col < a.N ? (col + half * a.up) * K + chunk * 16 : OOB;
      }
    }
    auto issue = [&](int st) {
      unsigned char* base = smem + A_BYTES + (st % NS) * STAGE;
      const bool last = st == nk - 1, past = st >= s_end;
#pragma unroll
      for (int q = 0; q < LPW; ++q) {
        const int ins = wave * LPW + q;  // wave-uniform
        auto* dst = (__attribute__((address_space(3))) void*)(base + ins * 1024);
        const int vo = voff[q] == OOB || past || (last && !((tail >> q) & 1)) ? OOB : voff[q] + st * ROWB;
        if (ins < A_INS) __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, dst, 16, vo, 0, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(b_rsrc, dst, 16, vo, 0, 0, BM <= 64 ? 2 : 0);
      }
    };
    typename Op::Acc acc[TM][NACC];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < NACC; ++j)
#pragma unroll
        for (int q = 0; q < Op::NR; ++q) acc[i][j][q] = 0;
    const int mb = min(TM, max(0, (m_rows - wm * WTM + S - 1) / S));  // blocks with rows (wave-uniform)
    const int sw = swizzle(fr);  // blocks start at multiples of 16 rows
    auto multiply = [&](int st) {
      const unsigned char* base = smem + A_BYTES + (st % NS) * STAGE + fr * ROWB;
      const unsigned char* few = smem + ((st - s_begin) * kFewRows + (fr & (kFewRows - 1))) * ROWB;
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        const int xo = ((ks * (Op::KS / 16) + fq) ^ sw) << 4;
        u32x4 fa[TM], fb[NACC];
#pragma unroll
        for (int j = 0; j < NACC; ++j) {
          const int r0 = SA + (GATED ? (j / TN) * OUTC + wn * WTN + (j % TN) * S : wn * WTN + j * S);
          fb[j] = ld16(base + r0 * ROWB + xo);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
          fa[i] = FEW ? ld16(few + (((ks * (Op::KS / 16) + fq) ^ swizzle(fr & (kFewRows - 1))) << 4))
                      : ld16(base + (wm * WTM + i * S) * ROWB + xo);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          if (i < mb) {
#pragma unroll
            for (int j = 0; j < NACC; ++j) Op::step(acc[i][j], fa[i], fb[j]);
          }
      }
    };
    wait_loads<0>();  // the scale and row lookups: the waits below count stage loads only
    if constexpr (PP) {
      constexpr int KPH = 2, PHASES = KSTEPS / KPH;  // K steps per phase, phases of a stage
      const int grp = wave >> 2;
      u32x4 frag[KPH][TM + NACC];
      auto phase_end = [&](bool wait) {
        if (wait) wait_loads<0>();
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      };
      auto phase = [&](int st, auto J) {
        constexpr int j = decltype(J)::value;
        // stage st + 1 goes where stage st - 1 was, which both groups finished reading before this phase
        if (j == 0 && st >= 1) issue(st + 1);
        const unsigned char* base = smem + (st & 1) * STAGE + fr * ROWB;
#pragma unroll
        for (int k = 0; k < KPH; ++k) {
          const int xo = (((j * KPH + k) * (Op::KS / 16) + fq) ^ sw) << 4;
#pragma unroll
          for (int i = 0; i < TM; ++i) frag[k][i] = ld16(base + (wm * WTM + i * S) * ROWB + xo);
#pragma unroll
          for (int n = 0; n < NACC; ++n) {
            const int r0 = BM + (GATED ? (n / TN) * OUTC + wn * WTN + (n % TN) * S : wn * WTN + n * S);
            frag[k][TM + n] = ld16(base + r0 * ROWB + xo);
          }
        }
        // stage st + 1 has to have landed when the group that runs first starts on it
        phase_end(j == PHASES - 1 && grp == 1);
        __builtin_amdgcn_s_setprio(1);
        if (mb > 0) {  // waves without rows save the power
#pragma unroll
          for (int k = 0; k < KPH; ++k)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
              for (int n = 0; n < NACC; ++n) Op::step(acc[i][n], frag[k][i], frag[k][TM + n]);
        }
        __builtin_amdgcn_s_setprio(0);
        phase_end(j == PHASES - 1 && grp == 0);
      };
      issue(0);
      issue(1);
      wait_loads<LPW>();
      lds_barrier();
      if (grp == 1) phase_end(false);
      for (int st = 0; st < nk; ++st) {
        phase(st, std::integral_constant<int, 0>{});
        phase(st, std::integral_constant<int, 1>{});
      }
      if (grp == 0) phase_end(false);
    } else {
#pragma unroll
      for (int i = 0; i < NS - 1; ++i) issue(s_begin + i);
      if constexpr (FEW) {
        // codes of the part's columns: 16 of a row per thread and round; past K they are zeros
        lds_barrier();  // the maxima
        const int units = m_rows * (s_end - s_begin) * 8;
        for (int u = tid; u < units; u += NTH) {
          const int r = u % m_rows, chunk = u / m_rows, c = s_begin * ROWB + chunk * 16;
          const I8Row row = i8_row(__float_as_uint(s_scale[r]));
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (c < K) {
            float v[16];
            const float* h = a.h + (int64_t)(p0 + r) * K + c;
#pragma unroll
            for (int q = 0; q < 4; ++q) unpack(ld16(h + 4 * q), *reinterpret_cast<float(*)[4]>(&v[4 * q]));
            i8_codes(v, row, w);
          }
          st16(smem + ((chunk >> 3) * kFewRows + r) * ROWB + (((chunk & 7) ^ swizzle(r)) << 4), u32x4{w[0], w[1], w[2], w[3]});
        }
        lds_barrier();
        if (tid < BM) s_scale[tid] = i8_row(__float_as_uint(s_scale[tid])).scale;
      }
      for (int st = s_begin; st < s_end; ++st) {
        wait_loads<(NS - 2) * LPW>();
        lds_barrier();  // stage st has landed for every wave, and stage st - 1 has been read
        issue(st + NS - 1);
        multiply(st);
      }
    }

    if constexpr (SPLIT && !GATED) {
      if (a.split > 1) {  // (uniform)
        constexpr int PV = TM * NACC * Op::NR / 2;  // pairs of sums per thread
        const int64_t slot = ((int64_t)tile * a.split + sp) * PV * NTH + tid;
        uint64_t* part = reinterpret_cast<uint64_t*>(a.partial);
#pragma unroll
        for (int v = 0; v < PV; ++v) {
          const int q = 2 * v, i = q / (NACC * Op::NR), j = q / Op::NR % NACC, n = q % Op::NR;
          __hip_atomic_store(part + slot + v * NTH,
                             (uint64_t)(uint32_t)acc[i][j][n] | ((uint64_t)(uint32_t)acc[i][j][n + 1] << 32),
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        // agent-scope stores write through to where every XCD reads them, so their acknowledgement is all the order that
        // the count needs. Nothing waits for another workgroup: the last to arrive finishes the tile. (The memory model's release
        // and acquire, which are for plain accesses that an L2 may hold, would write back and drop caches for every part: 38 us
        // instead of 26 for one Mixtral-shaped token's down pass.)
        int* s_last = reinterpret_cast<int*>(s_top);
        wait_loads<0>();
        lds_barrier();
        if (tid == 0)
          *s_last = __hip_atomic_fetch_add(a.ticket + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.split - 1;
        lds_barrier();
        if (!__builtin_amdgcn_readfirstlane(*s_last)) continue;
        for (int o = 0; o < a.split; ++o) {  // int32 sums: exact in any order
          if (o == sp) continue;
          const int64_t from = ((int64_t)tile * a.split + o) * PV * NTH + tid;
#pragma unroll
          for (int v = 0; v < PV; ++v) {
            const int q = 2 * v, i = q / (NACC * Op::NR), j = q / Op::NR % NACC, n = q % Op::NR;
            const uint64_t w = __hip_atomic_load(part + from + v * NTH, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            acc[i][j][n] += (int)(uint32_t)w;
            acc[i][j][n + 1] += (int)(uint32_t)(w >> 32);
          }
        }
      }
    }
    const int c_lane = n0 + wn * WTN + fr;  // column of block j: + j * S
    if constexpr (SPLIT && GATED) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int q = 0; q < Op::NR; ++q) {
          const int r = wm * WTM + i * S + Op::out_row(lane, q);
          if (r < m_rows) {
            int* o = a.partial + sp * a.partial_stride + (int64_t)(p0 + r) * a.w_rows;  // w_rows sums of a row
#pragma unroll
            for (int j = 0; j < TN; ++j)
              if (c_lane + j * S < a.N) {
                o[c_lane + j * S] = acc[i][j][q];
                o[a.up + c_lane + j * S] = acc[i][j + TN][q];
              }
          }
        }
    } else if constexpr (GATED) {
      float sg[TN], su[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int c = min(c_lane + j * S, a.N - 1);
        sg[j] = w_scale[c];
        su[j] = w_scale[a.up + c];
      }
      float* h = a.h + (int64_t)p0 * a.N;  // of the tile: 32-bit offsets from there
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i >= mb) break;  // no rows
#pragma unroll
        for (int q = 0; q < Op::NR; ++q) {
          const int r = wm * WTM + i * S + Op::out_row(lane, q);
          const float sr = s_scale[r];
          int top = 0;  // bits of |h|: positive, so they compare like integers
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const float v = silu((float)acc[i][j][q] * sr * sg[j]) * ((float)acc[i][j + TN][q] * sr * su[j]);
            const bool in = c_lane + j * S < a.N;
            if (in) top = max(top, (int)abs_bits(v));
            if (in && r < m_rows) h[r * a.N + c_lane + j * S] = v;
          }
          // over the 16 lanes of a DPP row, where they share r; the rest in LDS
          top = max(top, dpp_i32<0xB1>(top));
          top = max(top, dpp_i32<0x4E>(top));
          top = max(top, dpp_i32<0x141>(top));
          top = max(top, dpp_i32<0x140>(top));
          if ((lane & 15) == 0) s_top[(wn * (S / 16) + fr / 16) * BM + r] = top;
        }
      }
      lds_barrier();
      for (int r = tid; r < m_rows; r += NTH) {
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < WN * (S / 16); ++w) top = max(top, s_top[w * BM + r]);
        a.h_top[(int64_t)(p0 + r) * a.h_tiles + nt] = top;
      }
    } else {
      wait_loads<0>();
      lds_barrier();  // every wave is past its last stage, whose LDS takes the output tile
      float sd[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) sd[j] = w_scale[min(c_lane + j * S, a.N - 1)];
      constexpr int CPO = OUTC / 8;  // chunk c of output row r at c ^ (4 * ((r >> 2) & 1))
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int q = 0; q < Op::NR; ++q) {
          const int r = wm * WTM + i * S + Op::out_row(lane, q);
          const float sr = s_scale[r];
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const int c = wn * WTN + j * S + fr;
            *reinterpret_cast<bf16_t*>(smem + r * OUTC * 2 + (((c >> 3) ^ (((r >> 2) & 1) << 2)) << 4) + (c & 7) * 2) =
                (bf16_t)((float)acc[i][j][q] * sr * sd[j]);
          }
        }
      lds_barrier();
      for (int o = tid; o < BM * CPO; o += NTH) {
        const int r = o / CPO, ch = o % CPO, col = n0 + ch * 8;
        if (r < m_rows && col < a.N)
          st16(a.out + (int64_t)s_row[r] * a.N + col, ld16(smem + r * OUTC * 2 + ((ch ^ (((r >> 2) & 1) << 2)) << 4)));
      }
    }
  }
}

// Codes of h: a workgroup per row and 2048 columns. Every wave finds the row's maximum from its tiles' itself.
constexpr int kHCols = 2048;
__global__ __launch_bounds__(256) void i8_h_kernel(const float* __restrict__ h, const uint32_t* __restrict__ h_top,
                                                   int h_tiles, const int* __restrict__ total, int F,
                                                   int8_t* __restrict__ codes, float* __restrict__ scale) {
  const int rows = *total;
  const int c = blockIdx.x * kHCols + threadIdx.x * 8;
  for (int64_t p = blockIdx.y; p < rows; p += gridDim.y) {
    u32x4 lo{0u, 0u, 0u, 0u}, hi{0u, 0u, 0u, 0u};
    if (c < F) {
      lo = ld16_nt(h + p * F + c);
      hi = ld16_nt(h + p * F + c + 4);
    }
    uint32_t top = 0;
    for (int i = lane_id(); i < h_tiles; i += 64) top = max(top, h_top[p * h_tiles + i]);
    const I8Row r = i8_row(wave_top(top));
    if (blockIdx.x == 0 && threadIdx.x == 0) scale[p] = r.scale;
    if (c < F) {
      float v[8];
      unpack(lo, *reinterpret_cast<float(*)[4]>(&v[0]));
      unpack(hi, *reinterpret_cast<float(*)[4]>(&v[4]));
      uint32_t w[2];
      i8_codes(v, r, w);
      *reinterpret_cast<u32x2*>(codes + p * F + c) = u32x2{w[0], w[1]};
    }
  }
}

// The expert of plan row p: the last l with row_start[l] <= p
__device__ __forceinline__ int row_expert(const I8Args& a, int p) {
  int l = 0;
  for (int hi = a.El; hi - l > 1;) {
    const int mid = (l + hi) >> 1;
    if (a.row_start[mid] <= p) l = mid;
    else hi = mid;
  }
  return l;
}

// The parts of a split gate/up pass added (int32: exact in any order), and h as i8_gemm_kernel makes it: a wave per row and
// 64 columns, the tile of its maximum.
__global__ __launch_bounds__(256) void i8_sum_h_kernel(I8Args a) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int p = (int)(unit / a.h_tiles), tile = (int)(unit - (int64_t)p * a.h_tiles);
  if (p >= a.row_start[a.El]) return;
  const int c = tile * 64 + lane_id();
  const bool in = c < a.N;
  int g = 0, u = 0;
  for (int s = 0; s < a.split; ++s) {
    const int* o = a.partial + s * a.partial_stride + (int64_t)p * a.w_rows + (in ? c : 0);
    g += o[0];
    u += o[a.up];
  }
  const float sr = a.a_scale[a.a_perm ? a.a_perm[p] : p];
  const float* sw = a.w_scale + (int64_t)row_expert(a, p) * a.w_rows + (in ? c : 0);
  const float v = silu((float)g * sr * sw[0]) * ((float)u * sr * sw[a.up]);
  if (in) a.h[(int64_t)p * a.N + c] = v;
  const uint32_t top = wave_top(in ? abs_bits(v) : 0u);
  if (lane_id() == 0) a.h_top[(int64_t)p * a.h_tiles + tile] = top;
}

int i8_grid(int64_t tiles, int64_t most) {
  int64_t g = std::min(tiles, most);
  if (g >= 8) g &= ~7ll;
  return (int)std::max<int64_t>(g, 1);
}

constexpr int kPlanCus = 256;  // what a call is cut into is a function of its sizes alone, as its workspace is

// The tiles: rows, columns of h and of the output, workgroups per CU
struct I8Tile {
  int bm, gu_cols, dn_cols, per_cu, dn_per_cu;  // (down, 32 rows, Kimi-K2 decode: 120 us with two workgroups per CU, 113 with 3)
};
constexpr I8Tile kTiles[] = {{32, 64, 64, 2, 3}, {64, 64, 128, 2, 2}, {128, 128, 256, 1, 1}, {256, 128, 256, 1, 1}};

template <int I, typename Op, int WM, int WN, int GUNS, int DNNS, bool PP = false>
void launch_gemms(const I8Args& gu, const I8Args& dn, int64_t rows, int64_t mtiles, int num_cus, hipStream_t stream) {
  constexpr I8Tile t = kTiles[I];
  constexpr int NTH = WM * WN * 64, GUN = 2 * t.gu_cols, DNN = t.dn_cols;
  auto grid = [&](int64_t tiles) { return i8_grid(tiles, t.per_cu * num_cus); };
  const int64_t gu_tiles = mtiles * ceil_div_host(gu.N, t.gu_cols), dn_tiles = mtiles * ceil_div_host(dn.N, t.dn_cols);
  bool gu_split = false, dn_split = false;
  if constexpr (t.bm == 32) {
    gu_split = gu.split > 1;
    dn_split = dn.split > 1;
    if (gu_split) {
      i8_gemm_kernel<Op, t.bm, GUN, WM, WN, GUNS, t.per_cu, PP, true, true>
          <<<grid(gu_tiles * gu.split), NTH, 0, stream>>>(gu, (int)(rows * gu.K));
      i8_sum_h_kernel<<<(unsigned)ceil_div_host64(rows * gu.h_tiles, 4), 256, 0, stream>>>(gu);
    }
  }
  if (!gu_split)
    i8_gemm_kernel<Op, t.bm, GUN, WM, WN, GUNS, t.per_cu, PP, true>
        <<<grid(gu_tiles), NTH, 0, stream>>>(gu, (int)(rows * gu.K));
  if constexpr (t.bm == 32) {
    if (rows <= kFewRows) {
      i8_gemm_kernel<Op, 16, DNN, WM, WN, DNNS, t.per_cu, PP, false, true, true>
          <<<grid(dn_tiles * dn.split), NTH, 0, stream>>>(dn, 0);
      return;
    }
  }
  const dim3 hg(ceil_div_host(gu.N, kHCols), (unsigned)std::min<int64_t>(rows, 65535));
  i8_h_kernel<<<hg, 256, 0, stream>>>(gu.h, gu.h_top, gu.h_tiles, gu.row_start + gu.El, gu.N, const_cast<int8_t*>(dn.A),
                                      const_cast<float*>(dn.a_scale));
  if constexpr (t.bm == 32) {
    if (dn_split) {
      i8_gemm_kernel<Op, t.bm, DNN, WM, WN, DNNS, t.per_cu, PP, false, true>
          <<<grid(dn_tiles * dn.split), NTH, 0, stream>>>(dn, (int)(rows * dn.K));
    }
  }
  if (!dn_split)
    i8_gemm_kernel<Op, t.bm, DNN, WM, WN, DNNS, t.dn_per_cu, PP, false>
        <<<i8_grid(dn_tiles, t.dn_per_cu * num_cus), NTH, 0, stream>>>(dn, (int)(rows * dn.K));
}

// What a call is cut into: the tile, and for 32-row tiles the parts of each pass's K and the stages of a part.
struct I8Plan {
  int tile, gu_split, gu_stages, dn_split, dn_stages;
};

// Tiles of a row block count when the rows are spread evenly over the experts (hot experts, which a call's sizes do not show,
// have other counts); fewer rows than experts reach as many at most
int64_t row_tiles(int64_t rows_max, int El, int bm) {
  const int64_t n = std::min<int64_t>(El, rows_max);
  return n * ceil_div_host64(ceil_div_host64(rows_max, n), bm);
}

// The tile whose two passes take least, from the time of a round of stages: 2.3 us for 256 rows, 1.5 for 128, and for two
// workgroups per CU 1.32 (64 rows) and 0.89 (32 rows); a last round of one workgroup per CU takes 1.15 and 0.85. Whole MLPs (us)
// by rows of a tile, which this rule orders right but for ties:
//   experts, H, F, rows each      32      64     128     256
//   32, 7168, 2048, 32           242     244     272     339
//   32, 7168, 2048, 64           410     272     297     359
//   32, 7168, 2048, 128          752     461     340     382
//   32, 7168, 2048, 256         1476     822     521     450
//   8, 4096, 14336, 32           242     241     296     391
//   8, 4096, 14336, 96           611     506     348     428
//   12, 1184, 736, 64           27.9    27.1    32.5    43.2
//   12, 1184, 736, 128          40.3    34.8    38.5    45.6
//   12, 1184, 736, 384          79.7    62.2    46.3    55.3
//   16, 2048, 768, 128          51.1    40.6    44.1    51.8
//   48, 1024, 512, 96           53.7    47.9    40.3    47.6
double tile_cost(int i, int64_t rows_max, int El, int H, int F) {
  constexpr double full[] = {0.89, 1.32, 1.5, 2.3}, rest[] = {0.85, 1.15, 1.5, 2.3};
  const int64_t m = row_tiles(rows_max, El, kTiles[i].bm), slots = kTiles[i].per_cu * kPlanCus;
  auto pass = [&](int cols, int tile_cols, int K) {
    const int64_t tiles = m * ceil_div_host(cols, tile_cols), left = tiles % slots;
    return ceil_div_host(K, 128) * (tiles / slots * full[i] + (left == 0 ? 0.0 : left <= kPlanCus ? rest[i] : full[i]));
  };
  return pass(F, kTiles[i].gu_cols, H) + pass(H, kTiles[i].dn_cols, F);
}

// Parts of a pass's K with 32-row tiles: as many as give every CU its workgroups, of at least 8 stages each, as the parts' sums
// take a launch of their own (gate/up) or a wait for the last part; at most `most` stages.
void split_k(int64_t tiles, int K, int most, int& split, int& stages) {
  const int nk = ceil_div_host(K, 128);
  split = (int)std::max<int64_t>(ceil_div_host(nk, most), std::min<int64_t>(kTiles[0].per_cu * kPlanCus / tiles, nk / 8));
  stages = ceil_div_host(nk, split);
  split = ceil_div_host(nk, stages);  // every part has stages
}

I8Plan i8_plan(int64_t rows_max, int El, int H, int F) {
  I8Plan p{0, 1, 0, 1, 0};
  if (rows_max == 0) return p;
  for (int i = 1; i < 4 && rows_max > kFewRows; ++i)
    if (tile_cost(i, rows_max, El, H, F) < tile_cost(p.tile, rows_max, El, H, F)) p.tile = i;
  if (p.tile == 0) {
    const int64_t m = row_tiles(rows_max, El, 32);
    split_k(m * ceil_div_host(F, kTiles[0].gu_cols), H, 1 << 30, p.gu_split, p.gu_stages);
    split_k(m * ceil_div_host(H, kTiles[0].dn_cols), F, rows_max <= kFewRows ? kFewStages : 1 << 30, p.dn_split, p.dn_stages);
  }
  return p;
}

int h_tiles(const I8Plan& p, int F) { return ceil_div_host(F, kTiles[p.tile].gu_cols); }

// the workspace: plan, row map, h, its tiles' maxima, its codes and scales, the parts of a split pass (gate/up's are
// done with before the down pass writes its own) and the down tiles' tickets
struct I8Scratch {
  size_t plan, perm, h, top, codes, scale, partial, ticket, total;
  int tickets;
};
int64_t row_tiles_most(int64_t rows, int El, int bm) { return ceil_div_host64(rows, bm) + std::min<int64_t>(El, rows); }
I8Scratch i8_scratch(int64_t rows, int El, int H, int F, const I8Plan& p) {
  I8Scratch s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  s.plan = take(mlp_plan_ints(El) * sizeof(int));
  s.perm = take((size_t)rows * sizeof(int));
  s.h = take((size_t)rows * (size_t)F * sizeof(float));
  s.top = take((size_t)rows * (size_t)h_tiles(p, F) * sizeof(uint32_t));
  s.codes = take((size_t)rows * (size_t)F);
  s.scale = take((size_t)rows * sizeof(float));
  // down: 32 x 64 sums a tile and part
  const int64_t dn_tiles = p.dn_split > 1 ? row_tiles_most(rows, El, 32) * ceil_div_host(H, kTiles[0].dn_cols) : 0;
  s.tickets = (int)dn_tiles;
  s.partial = take(std::max(p.gu_split > 1 ? (size_t)p.gu_split * 2 * (size_t)F * (size_t)rows : 0,
                            (size_t)dn_tiles * p.dn_split * 32 * kTiles[0].dn_cols) * sizeof(int));
  s.ticket = take((size_t)s.tickets * sizeof(int));
  s.total = at;
  return s;
}

}  // namespace

// Rows of either pass and one expert's weights are addressed by 31-bit byte offsets; K products of codes of either sign
// (128 * 128 at most) stay within an int32 sum
bool mlp_i8_fits(int64_t rows, int H, int F) {
  return std::max(H, F) < 1 << 17 && rows * std::max<int64_t>(H, F) < 0x7ffffe00ll &&
         2 * (int64_t)F * H < 0x7ffffe00ll;
}

I8Tiling mlp_i8_tiling(int64_t rows, int El, int H, int F) {
  const I8Plan p = i8_plan(rows, El, H, F);
  return {kTiles[p.tile].bm, p.gu_split, p.dn_split};
}

size_t mlp_i8_workspace_bytes(int64_t rows, int El, int H, int F) {
  return i8_scratch(rows, El, H, F, i8_plan(rows, El, H, F)).total;
}

hipError_t launch_expert_mlp_i8(const int8_t* send_q, const float* send_scale, const moe_layout_t& L,
                                const int8_t* gu_codes, const float* gu_scales, const int8_t* dn_codes,
                                const float* dn_scales, int F, void* out_buf, void* workspace, int num_cus,
                                hipStream_t stream) {
  const int El = L.E / L.R;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (rows == 0) return hipSuccess;
  const I8Plan p = i8_plan(rows, El, L.H, F);
  const I8Scratch at = i8_scratch(rows, El, L.H, F, p);
  char* ws = static_cast<char*>(workspace);
  int* plan = reinterpret_cast<int*>(ws + at.plan);
  int* perm = reinterpret_cast<int*>(ws + at.perm);
  // with one rank the send rows are in plan order and the offsets are the row starts: no plan is needed
  const bool ranks = L.R > 1;
  if (ranks) launch_mlp_plan(L, kTiles[p.tile].bm, plan, perm, stream);
  const int* row_start = ranks ? plan + 2 : L.expert_offset;
  const int* tile_start = ranks ? plan + 3 + El : nullptr;
  I8Args gu{};
  gu.A = send_q;
  gu.a_perm = ranks ? perm : nullptr;
  gu.a_scale = send_scale;
  gu.W = gu_codes;
  gu.w_scale = gu_scales;
  gu.K = L.H;
  gu.N = F;
  gu.w_rows = 2 * F;
  gu.up = F;
  gu.h = reinterpret_cast<float*>(ws + at.h);
  gu.h_top = reinterpret_cast<uint32_t*>(ws + at.top);
  gu.h_tiles = h_tiles(p, F);
  gu.split = p.gu_split;
  gu.split_stages = p.gu_stages;
  gu.partial = reinterpret_cast<int*>(ws + at.partial);
  gu.partial_stride = rows * 2 * F;
  gu.zero = reinterpret_cast<int*>(ws + at.ticket);
  gu.zero_n = at.tickets;
  gu.row_start = row_start;
  gu.tile_start = tile_start;
  gu.El = El;
  I8Args dn{};
  dn.A = reinterpret_cast<int8_t*>(ws + at.codes);
  dn.a_scale = reinterpret_cast<float*>(ws + at.scale);
  dn.W = dn_codes;
  dn.w_scale = dn_scales;
  dn.K = F;
  dn.N = L.H;
  dn.w_rows = L.H;
  dn.out = static_cast<bf16_t*>(out_buf);
  dn.out_perm = ranks ? perm : nullptr;
  dn.row_start = row_start;
  dn.tile_start = tile_start;
  dn.El = El;
  dn.split = p.dn_split;
  dn.split_stages = p.dn_stages;
  dn.partial = reinterpret_cast<int*>(ws + at.partial);
  dn.ticket = reinterpret_cast<int*>(ws + at.ticket);
  dn.h = gu.h;
  dn.h_top = gu.h_top;
  dn.h_tiles = gu.h_tiles;
  const int64_t mtiles = row_tiles_most(rows, El, kTiles[p.tile].bm);
  if (p.tile == 0) launch_gemms<0, OpI16, 1, 4, 3, 4>(gu, dn, rows, mtiles, num_cus, stream);
  else if (p.tile == 1) launch_gemms<1, OpI32, 2, 2, 3, 3>(gu, dn, rows, mtiles, num_cus, stream);
  else if (p.tile == 2) launch_gemms<2, OpI32, 2, 4, 3, 3>(gu, dn, rows, mtiles, num_cus, stream);
  else launch_gemms<3, OpI32, 4, 2, 2, 2, true>(gu, dn, rows, mtiles, num_cus, stream);
  return hipGetLastError();
}

}  // namespace moe
