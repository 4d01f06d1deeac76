// Expert SwiGLU MLP on dispatched rows with 4-bit expert weights (moe_expert_mlp_w4).
//
// The plan (rows grouped by local expert, mlp.hip) and the two passes are moe_expert_mlp's: gate/up with
// h = silu(g) * u, then down. The weights are the M operand of the matrix unit (blocks of 16 output columns) and the
// rows its N operand, so a packed code tile, one contiguous kilobyte, is decoded in registers right into the
// operand it is (w4.h), and a lane ends up with four consecutive output columns of one row.
//
//   w4_gemm_kernel  BM rows x 64 WN weight rows per tile on v_mfma_f32_32x32x16_bf16. Rows go to LDS directly; the
//                   codes go from memory to the registers of the wave that multiplies them and never pass LDS.
//                   BM = 32 (four waves, four or three workgroups per CU) streams the codes of experts with few rows and
//                   is bound by their bytes; BM = 128 and 256 (eight waves, one workgroup per CU) decode a code for more
//                   rows: at 1024 rows per expert the matrix units are busy 53 to 57 % of the cycles, at 100 to 250
//                   neither they nor the bytes are reached (1.4 to 1.9 times the longer of the two).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "mfma.h"
#include "tiles.h"
#include "w4.h"

namespace moe {

namespace {

struct W4Args {
  const bf16_t* A;       // rows [., K]: the send buffer, or h in plan order
  int64_t part;          // elements from A to its second part (h's remainders), 0 without one
  const int* a_perm;     // source row of a plan row, or nullptr (A in plan order)
  const uint8_t* codes;  // packed [El, N_w, K]
  const uint8_t* scales;
  int K, N;              // N: output columns (F or H)
  int w_rows;            // weight rows per expert (2F or H)
  int up;                // weight row of the up half (gate/up only)
  bf16_t* Out;           // [., N]
  int64_t out_part;      // elements from Out to the second part of h
  const int* out_perm;   // destination row of a plan row, or nullptr
  const int* plan;
  int El;
  // SPLIT: K in `split` parts of split_stages stages (a multiple of 8) each, their fp32 sums to partial [split, rows, N]
  int split, split_stages;
  float* partial;
  int64_t partial_stride;  // elements of one part
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// ------------------------------------------------------------------------------------------------
// the GEMM
// ------------------------------------------------------------------------------------------------
// BM rows x 64 WN weight rows per tile; WM x WN waves, each BM / WM rows x 64 weight rows: the gate and the up rows of 32
// columns of h, or 64 down rows. K goes in stages of 64:
//  - rows: 128 bytes each, straight to LDS, NS slots. 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7), so that a
//    fragment read touches every bank once.
//  - codes: one 16-byte load per lane and 32 weight rows holds a stage (lane % 32 the row, lane / 32 one of its two
//    scale groups). Its word j is the fragment of matrix step j, whose k are 8 j on of both groups; the row fragments
//    follow that order.
//  - scales: the tiles of eight stages go to LDS of the wave's own in one load, eight stages ahead (a load of a byte per
//    stage and row keeps the load path as long as one of sixteen).
//  - schedule: the weights of step j + 1 are decoded and its rows read while step j is multiplied. The barrier that
//    publishes stage s + 1 sits before the last step of stage s, whose fragments are in registers: after it the
//    slot of stage s is free and takes the rows of stage s + NS. Loads past the last stage are issued too, at offsets
//    that read nothing, so at least as many are in flight at every wait as it counts on.
// PARTS: h has two bf16 parts (16 significant bits) where few rows make the weights' bytes the bound, so that the
// down pass's doubled matrix work is free, and one where the matrix units are the bound.
// SPLIT: the down pass with K cut over workgroups, where its tiles are few and its K long (see w4_split).
template <int BM, int WM, int WN, bool GATED, int PARTS, bool SPLIT = false>
__global__ __launch_bounds__(WM * WN * 64, BM == 32 ? 4 : 1) void w4_gemm_kernel(W4Args a, int a_bytes) {
  static_assert(!SPLIT || !GATED, "the gate/up pass is not split");
  constexpr int NW = WM * WN, NTH = NW * 64, S = 32, NS = 4;
  constexpr int WTM = BM / WM, TM = WTM / S;
  constexpr int XP = GATED ? 1 : PARTS, OP = GATED ? PARTS : 1;  // parts of the rows read and written
  constexpr int STAGE = XP * BM * 128, XI = XP * BM / 8 / NW;    // bytes of a stage; 1 KB row loads per wave
  constexpr int OUTC = WN * (GATED ? 32 : 64);
  constexpr int OUT_BYTES = BM * OUTC * 2;
  constexpr int BODY = NS * STAGE > OP * OUT_BYTES ? NS * STAGE : OP * OUT_BYTES;
  constexpr int LOADS = XI + 2;  // loads per wave and stage: rows and codes
  // stages of codes in flight: three are what the registers leave next to 128 accumulators, and enough where several
  // workgroups share a CU; the 128-row tiles run alone on theirs, often with few tiles to hide a miss behind
  constexpr int CS = BM == 128 ? 6 : 3;
  constexpr int XB = BM == 256 ? 1 : 2;      // buffers of row fragments
  constexpr int OOB = 0x7ffffff0;
  static_assert(PARTS == 1 || WM == 1, "parts share a matrix step within one wave row");
  static_assert(TM >= 1 && XP * BM / 8 % NW == 0 && OUTC >= 128, "tile");
  // the only LDS object (a second one makes the compiler wait for every load in flight before LDS reads): the
  // stages, which the output tile reuses, then its destination rows, the waves' scales, the
  // plan's starts
  __shared__ __attribute__((aligned(1024))) unsigned char smem[BODY + BM * 4 + NW * 2048 + 2 * (MOE_MAX_EXPERTS + 1) * 4];
  int tid = threadIdx.x, lane = tid & 63;  // made opaque at each tile start (below)
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int fr = lane & 31, fq = lane >> 5;
  const int K = a.K, nk = (K + 63) / 64;
  const int kc = (K + W4_TILE_K - 1) / W4_TILE_K, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
  // the plan's row and tile starts in LDS: a search through memory costs a microsecond per step at each tile
  int* row_start = reinterpret_cast<int*>(smem + BODY + BM * 4 + NW * 2048);
  int* tile_start = row_start + MOE_MAX_EXPERTS + 1;
  for (int i = tid; i <= a.El; i += NTH) {
    row_start[i] = a.plan[2 + i];
    tile_start[i] = a.plan[3 + a.El + i];
  }
  const int n_tiles = (a.N + OUTC - 1) / OUTC;
  const Tiles mine = my_tiles(a.plan[0] * n_tiles * (SPLIT ? a.split : 1));
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.A, (short)0, a_bytes, 0x00020000);
  lds_barrier();
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
    // the two 32-row weight blocks (N % 32 == 0: a block is whole or past N, then it repeats the first rows): a
    // wave-uniform start, and the lane's offset from there
    const int c0 = nt * OUTC + wn * (GATED ? 32 : 64);
    const bool on[2] = {c0 < a.N, GATED ? c0 < a.N : c0 + 32 < a.N};
    const uint8_t* wc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t rb = ((int64_t)l * a.w_rows + (on[b] ? c0 + b * (GATED ? a.up : 32) : 0)) >> 4;
      wc[b] = a.codes + rb * kc * W4_CODE_TILE;
    }
    const uint32_t c_off = (uint32_t)((fr >> 4) * kc * W4_CODE_TILE + (fr & 15) * 16 + fq * 256);
    // this lane's row and 16-byte chunk in each of the wave's row loads
    int voff[XI];
#pragma unroll
    for (int q = 0; q < XI; ++q) {
      const int r = ((wave * XI + q) * 8 + (lane >> 3)) % BM;
      const int p = p0 + min(r, m_rows - 1);
      voff[q] = a.a_perm ? a.a_perm[p] : p;
    }
    u32x4 cw[CS][2];
    auto load_codes = [&](int st, int u) {
      const int s = min(st, nk - 1);
#pragma unroll
      for (int b = 0; b < 2; ++b) cw[u][b] = ld16(wc[b] + ((s >> 1) * W4_CODE_TILE + (s & 1) * 512) + c_off);
    };
    // the first codes are requested while the row lookups are on their way
    auto fence = [] { asm volatile("" ::: "memory"); };
    fence();
#pragma unroll
    for (int u = 0; u < CS - 3; ++u) load_codes(s_begin + u, u);
    fence();
#pragma unroll
    for (int q = 0; q < XI; ++q) {
      const int v = (wave * XI + q) * 8 + (lane >> 3), r = v % BM;
      voff[q] = r < m_rows ? (voff[q] * K + (v >= BM ? (int)a.part : 0)) * 2 + (((lane & 7) ^ ((r >> 1) & 7)) << 4) : OOB;
    }
    // bit q: this lane's chunk of load q lies within K in the last stage
    int tail = 0;
#pragma unroll
    for (int q = 0; q < XI; ++q) {
      const int r = ((wave * XI + q) * 8 + (lane >> 3)) % BM;
      tail |= ((nk - 1) * 64 + (((lane & 7) ^ ((r >> 1) & 7)) << 3) < K ? 1 : 0) << q;
    }
    auto load_rows = [&](int st) {
      unsigned char* base = smem + (st % NS) * STAGE + wave * XI * 1024;
#pragma unroll
      for (int q = 0; q < XI; ++q) {
        const bool in = st < nk - 1 || (st < nk && ((tail >> q) & 1));
        const int vo = in && voff[q] != OOB ? voff[q] + st * 128 : OOB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (__attribute__((address_space(3))) void*)(base + q * 1024), 16,
                                                 vo, 0, 0, 0);
      }
    };
    // scale tiles q of the wave's four 16-row blocks (1 KB) to its LDS, slot q & 1
    unsigned char* s_sc = smem + BODY + BM * 4 + wave * 2048;
    const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.scales + (int64_t)l * (a.w_rows >> 4) * ks * W4_SCALE_TILE), (short)0,
        (a.w_rows >> 4) * ks * W4_SCALE_TILE, 0x00020000);
    const int s_off = (((on[fq] ? c0 + fq * (GATED ? a.up : 32) : 0) >> 4) + (fr >> 4)) * ks * W4_SCALE_TILE + (fr & 15) * 16;
    auto load_scales = [&](int q) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s_rsrc, (__attribute__((address_space(3))) void*)(s_sc + (q & 1) * 1024), 16,
                                               s_off + min(q, ks - 1) * W4_SCALE_TILE, 0, 0, 0);
    };
    float sc[2];
    auto stage_scales = [&](int st) {
      const unsigned char* p = s_sc + ((st >> 3) & 1) * 1024 + (fr >> 4) * 256 + ((fr & 15) + 16 * fq) * 4 +
                               (st & 1) * 128 + ((st >> 1) & 3);
#pragma unroll
      for (int b = 0; b < 2; ++b) sc[b] = w4_scale(p[b * 512]);
    };
    f32x16 acc[TM][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][b][q] = 0.f;
    const int mb = min(TM, max(0, (m_rows - wm * WTM + S - 1) / S));  // blocks with rows (wave-uniform)

    wait_loads<0>();
    lds_barrier();  // the previous tile's output has left LDS
    // With two parts and at most 16 rows, both parts share a matrix step: its columns 0 .. 15 are the rows' first
    // parts and 16 .. 31 their second ones, which the epilogue adds up.
    const bool packed = XP == 2 && m_rows <= 16;
    const unsigned char* frag_base = smem + (packed ? (fr >> 4) * BM + (fr & 15) : wm * WTM + fr) * 128;
    const int sw = (fr >> 1) & 7;
    u32x4 xf[XB][XP][TM], wf[2][2];
    auto read_row = [&](int st, int j, int x, int i) {
      xf[j & (XB - 1)][x][i] = ld16(frag_base + (st % NS) * STAGE + (x * BM + i * S) * 128 + (((fq * 4 + j) ^ sw) << 4));
    };
    // the waits count loads: these groups must be issued in this order
    load_scales(s_begin >> 3);
    load_scales((s_begin >> 3) + 1);
    fence();
    load_rows(s_begin);
    fence();
    load_codes(s_begin + CS - 3, CS - 3);
    load_rows(s_begin + 1);
    fence();
    load_codes(s_begin + CS - 2, CS - 2);
    load_rows(s_begin + 2);
    fence();
    load_codes(s_begin + CS - 1, CS - 1);
    load_rows(s_begin + 3);
    wait_loads<2 * LOADS>();
    lds_barrier();
    stage_scales(s_begin);
#pragma unroll
    for (int x = 0; x < XP; ++x)
#pragma unroll
      for (int i = 0; i < TM; ++i) read_row(s_begin, 0, x, i);
#pragma unroll
    for (int b = 0; b < 2; ++b) wf[0][b] = w4_to_bf16(cw[0][b][0], sc[b]);
    auto stage = [&](int s, auto U) {
      constexpr int u = decltype(U)::value, un = (u + 1) % CS;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < 3) {
#pragma unroll
          for (int b = 0; b < 2; ++b) wf[(j + 1) & 1][b] = w4_to_bf16(cw[u][b][j + 1], sc[b]);
        } else {
          wait_loads<2 * LOADS>();  // stage s + 1 has landed: at most its two successors are in flight
          lds_barrier();
          load_codes(s + CS, u);
          load_rows(s + NS);
          if (((s + 1) & 7) == 0) load_scales(((s + 1) >> 3) + 1);
          stage_scales(s + 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) wf[0][b] = w4_to_bf16(cw[un][b][0], sc[b]);
        }
        // the next step's row fragments: before this step's products where there are registers for two sets, else
        // each as soon as this step has used it
        if constexpr (XB == 2) {
#pragma unroll
          for (int x = 0; x < XP; ++x)
#pragma unroll
            for (int i = 0; i < TM; ++i) read_row(j < 3 ? s : s + 1, (j + 1) & 3, x, i);
        }
#pragma unroll
        for (int x = 0; x < XP; ++x)
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            if (i < mb && !(x == 1 && packed)) {
              const u32x4 b[1] = {xf[j & (XB - 1)][x][i]};
              const u32x4 w0[1] = {wf[j & 1][0]}, w1[1] = {wf[j & 1][1]};
              Op32::step(acc[i][0], w0, b);
              Op32::step(acc[i][1], w1, b);
            }
            if constexpr (XB == 1) read_row(j < 3 ? s : s + 1, (j + 1) & 3, x, i);
          }
      }
    };
    for (int s = s_begin; s < s_end; s += CS) {
      stage(s, std::integral_constant<int, 0>{});
      if (s + 1 < s_end) stage(s + 1, std::integral_constant<int, 1>{});
      if (s + 2 < s_end) stage(s + 2, std::integral_constant<int, 2>{});
      if constexpr (CS > 3) {
        if (s + 3 < s_end) stage(s + 3, std::integral_constant<int, 3>{});
        if (s + 4 < s_end) stage(s + 4, std::integral_constant<int, 4>{});
        if (s + 5 < s_end) stage(s + 5, std::integral_constant<int, 5>{});
      }
    }
    // epilogue through LDS: lane l holds row l % 32 of a block and four consecutive columns per group of registers
    // (Op32::out_row); 16-byte chunk c of output row r sits at c ^ (r & 15)
    wait_loads<0>();
    lds_barrier();
    if (packed) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[0][b][q] = join_parts(acc[0][b][q], __shfl_xor(acc[0][b][q], 16, 64));
    }
    if constexpr (SPLIT) {
      // lane l holds row l % 32 of a block and four consecutive columns per group of registers
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = wm * WTM + i * S + fr;
        if (r < m_rows) {
          float* o = a.partial + sp * a.partial_stride + (int64_t)(p0 + r) * a.N + c0 + 4 * fq;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              if (on[b]) {
                const float v[4] = {acc[i][b][4 * q4], acc[i][b][4 * q4 + 1], acc[i][b][4 * q4 + 2], acc[i][b][4 * q4 + 3]};
                st16(o + b * 32 + 8 * q4, pack(v));
              }
        }
      }
      continue;
    }
    int* s_orow = reinterpret_cast<int*>(smem + BODY);
    for (int r = tid; r < BM; r += NTH) {
      const int p = p0 + min(r, m_rows - 1);
      s_orow[r] = a.out_perm ? a.out_perm[p] : p;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * WTM + i * S + fr;
#pragma unroll
      for (int b = 0; b < (GATED ? 1 : 2); ++b)
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          float v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = GATED ? silu(acc[i][0][4 * q4 + q]) * acc[i][1][4 * q4 + q] : acc[i][b][4 * q4 + q];
          const int chunk = (wn * (GATED ? 32 : 64) + b * 32) / 8 + q4;
          unsigned char* o = smem + r * OUTC * 2 + ((chunk ^ (r & 15)) << 4) + fq * 8;
          *reinterpret_cast<u32x2*>(o) = u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
          if constexpr (OP == 2) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = bf16_rest(v[q]);
            *reinterpret_cast<u32x2*>(o + OUT_BYTES) = u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
          }
        }
    }
    lds_barrier();
    constexpr int CPO = OUTC / 8;
    for (int o = tid; o < OP * BM * CPO; o += NTH) {
      const int v = o / CPO, chunk = o % CPO, r = v % BM, part = v / BM;
      if (r < m_rows && nt * OUTC + chunk * 8 < a.N)
        st16(a.Out + (part ? a.out_part : 0) + (int64_t)s_orow[r] * a.N + nt * OUTC + chunk * 8,
             ld16(smem + part * OUT_BYTES + r * OUTC * 2 + ((chunk ^ (r & 15)) << 4)));
    }
  }
}

// The parts of a split down pass added in order, rounded once and put into their rows: eight columns per thread.
__global__ __launch_bounds__(256) void w4_sum_kernel(const float* __restrict__ partial, int split, int64_t stride,
                                                     const int* __restrict__ plan, const int* __restrict__ perm, int N,
                                                     bf16_t* __restrict__ out) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  const int64_t p = at / N;
  if (p >= plan[1]) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < split; ++s) {
    float lo[4], hi[4];
    unpack(ld16(partial + s * stride + at), lo);
    unpack(ld16(partial + s * stride + at + 4), hi);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] += lo[q];
      v[4 + q] += hi[q];
    }
  }
  st16(out + (int64_t)perm[p] * N + (at - p * N), pack(v));
}

int w4_grid(int64_t tiles, int64_t most) {
  int64_t g = std::min(tiles, most);
  if (g >= 8) g &= ~7ll;
  return (int)std::max<int64_t>(g, 1);
}

// Workgroups that stay resident on a CU with 32-row tiles. Gate/up: four of 123 registers (and 28 KB of LDS; without the
// bound of four waves per SIMD the compiler takes 132). Down: three, of 45 KB of LDS. Whole passes with the grids and the
// split for four each while only three were resident, and as it is (us): 8 experts of 16 rows, H 4096, F 14336 194 ->
// 182, of 64 rows 313 -> 305; 3 experts of 1248 rows, H 224, F 10752 186 -> 170-176.
constexpr int kPerCuGateUp32 = 4, kPerCuDown32 = 3;
template <int BM, int WM, int WN, int PARTS>
void launch_gemms(const W4Args& gu, const W4Args& dn, int64_t rows, int64_t mtiles, int num_cus, hipStream_t stream) {
  constexpr int GU_PER_CU = BM == 32 ? kPerCuGateUp32 : 1, DN_PER_CU = BM == 32 ? kPerCuDown32 : 1, NTH = WM * WN * 64;
  w4_gemm_kernel<BM, WM, WN, true, PARTS>
      <<<w4_grid(mtiles * ceil_div_host(gu.N, WN * 32), GU_PER_CU * num_cus), NTH, 0, stream>>>(gu, (int)(rows * gu.K * 2));
  const int a_bytes = (int)((PARTS == 2 ? dn.part * 2 : 0) + rows * dn.K * 2);
  const int64_t tiles = mtiles * ceil_div_host(dn.N, WN * 64);
  if constexpr (BM == 32) {
    if (dn.split > 1) {
      w4_gemm_kernel<BM, WM, WN, false, PARTS, true>
          <<<w4_grid(tiles * dn.split, DN_PER_CU * num_cus), NTH, 0, stream>>>(dn, a_bytes);
      w4_sum_kernel<<<(unsigned)ceil_div_host64(rows * dn.N / 8, 256), 256, 0, stream>>>(
          dn.partial, dn.split, dn.partial_stride, dn.plan, dn.out_perm, dn.N, dn.Out);
      return;
    }
  }
  w4_gemm_kernel<BM, WM, WN, false, PARTS><<<w4_grid(tiles, DN_PER_CU * num_cus), NTH, 0, stream>>>(dn, a_bytes);
}

// Parts of the down pass's K with 32-row tiles: as many as give every CU its three workgroups, of 16 stages at least, and
// no more than F / H, so that the parts' sums take no more workspace than h's two parts. 8 experts of 16 rows, H 4096,
// F 14336 (128 tiles of 224 stages): the whole pass 233 -> 181 us; 4 experts of 16 rows, H 512, F 8192: 78 -> 32 us, of
// 256 rows: 113 -> 68 us; 3 experts of 1248 rows, H 224, F 10752: 211 -> 170 us.
// Only up to 128 tiles of rows, as the workspace leaves room for the sums without knowing H.
constexpr int kSplitMaxTiles = 128;
int64_t row_tiles32(int64_t rows_max, int El) { return El * ceil_div_host64(ceil_div_host64(rows_max, El), 32); }
int w4_split(int64_t rows_max, int El, int H, int F, int num_cus) {
  if (row_tiles32(rows_max, El) > kSplitMaxTiles) return 1;
  const int64_t tiles = row_tiles32(rows_max, El) * ceil_div_host(H, 256);
  const int64_t s = std::min<int64_t>({kPerCuDown32 * num_cus / tiles, F / H, F / 64 / 16});
  return s < 2 ? 1 : (int)s;
}

// Rows per M tile, by the time both passes would take with each, from the largest tile counts the capacity allows. A
// round of 256-row tiles, one per CU, is the unit for every k; a round of 128-row tiles takes 0.57 of it. 32-row tiles
// wait on memory, not on the matrix units, and share a CU: each of a full round's takes 0.28, and those of the last one
// 0.22 and 0.1 together.
// Whole passes (us):
//   experts, H, F, rows each      32     128     256
//   32, 7168, 2048, 32           193     253     376
//   32, 7168, 2048, 64           287     292     394
//   32, 7168, 2048, 96           407     346     432
//   32, 7168, 2048, 192          722     656     569
//   8, 4096, 14336, 96           414     403     519
//   8, 4096, 14336, 256          931     713     772
//   4, 2048, 1024, 256            41      58      90
//   4, 2048, 1024, 512            53      62      93
//   4, 2048, 1024, 1024           85      68     100
//   16, 2048, 768, 100            48      57      69
//   16, 2048, 768, 200            67      62      87
//   8, 2048, 2048, 128            57      72      88
//   8, 288, 2016, 640             71      74      99
//   8, 288, 2016, 1280           119     101     123
//   12, 1184, 736, 256            46      49      74
// (64-row tiles with two workgroups per CU were never more than 8 % better than the best of these, and often worse.)
int w4_rows(int64_t rows_max, int El, int H, int F, int num_cus) {
  const int64_t per = ceil_div_host64(rows_max, El);
  auto rounds = [&](int bm, int64_t n_tiles, int per_cu32) {
    const double t = (double)El * ceil_div_host64(per, bm) * n_tiles / num_cus;  // tiles per CU
    if (bm == 256) return std::ceil(t);
    if (bm == 128) return 0.57 * std::ceil(t);
    const double full = std::floor(t / per_cu32), rest = t - per_cu32 * full;
    return full * 0.28 * per_cu32 + (rest > 0 ? 0.1 + 0.22 * rest : 0.0);
  };
  auto cost = [&](int bm, int split) {
    return H * rounds(bm, ceil_div_host(F, 128), kPerCuGateUp32) +
           (double)F / split * rounds(bm, (int64_t)ceil_div_host(H, 256) * split, kPerCuDown32);
  };
  const double c32 = cost(32, w4_split(rows_max, El, H, F, num_cus)), c128 = cost(128, 1), c256 = cost(256, 1);
  if (c32 <= c128 && c32 <= c256) return 32;
  return c128 <= c256 ? 128 : 256;
}

}  // namespace

W4Tiling mlp_w4_tiling(int64_t rows, int El, int H, int F, int num_cus) {
  if (rows == 0) return {32, 1, 0};  // nothing runs
  W4Tiling t{w4_rows(rows, El, H, F, num_cus), 1, 0};
  if (t.rows == 32) {
    const int nk = ceil_div_host(F, 64);
    t.parts = w4_split(rows, El, H, F, num_cus);
    t.stages = (ceil_div_host(nk, t.parts) + 7) & ~7;
    t.parts = ceil_div_host(nk, t.stages);  // every part has stages
  }
  return t;
}

// Rows of either pass, one expert's scales and a 16-row block's codes are addressed by 31-bit byte offsets
bool mlp_w4_fits(int64_t rows, int H, int F) {
  auto scales = [](int64_t n, int64_t k) { return n / 16 * ceil_div_host64(k, W4_STILE_K) * W4_SCALE_TILE; };
  return rows * std::max<int64_t>(H, 2 * (int64_t)F) * 2 < 0x7ffffe00ll && std::max(H, F) < 1 << 27 &&
         std::max(scales(2 * (int64_t)F, H), scales(H, F)) <= INT32_MAX;
}

size_t mlp_w4_workspace_bytes(int64_t rows, int El, int F) {
  return align256(mlp_plan_ints(El) * sizeof(int)) + align256((size_t)rows * sizeof(int)) +
         2 * align256((size_t)rows * (size_t)F * 2) +
         (row_tiles32(rows, El) <= kSplitMaxTiles ? align256((size_t)rows * (size_t)F * 4) : 0);
}

hipError_t launch_expert_mlp_w4(const void* send_buf, const moe_layout_t& L, const uint8_t* gu_codes,
                                const uint8_t* gu_scales, const uint8_t* dn_codes, const uint8_t* dn_scales, int F,
                                void* out_buf, void* workspace, int num_cus, hipStream_t stream) {
  const int El = L.E / L.R;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (rows == 0) return hipSuccess;
  char* ws = static_cast<char*>(workspace);
  int* plan = reinterpret_cast<int*>(ws);
  ws += align256(mlp_plan_ints(El) * sizeof(int));
  int* perm = reinterpret_cast<int*>(ws);
  ws += align256((size_t)rows * sizeof(int));
  bf16_t* h = reinterpret_cast<bf16_t*>(ws);
  const int64_t h_part = (int64_t)(align256((size_t)rows * (size_t)F * 2) / 2);
  const W4Tiling tiling = mlp_w4_tiling(rows, El, L.H, F, num_cus);
  const int bm = tiling.rows;
  launch_mlp_plan(L, bm, plan, perm, stream);
  W4Args gu{};
  gu.A = static_cast<const bf16_t*>(send_buf);
  gu.a_perm = perm;
  gu.codes = gu_codes;
  gu.scales = gu_scales;
  gu.K = L.H;
  gu.N = F;
  gu.w_rows = 2 * F;
  gu.up = F;
  gu.Out = h;
  gu.out_part = h_part;
  gu.plan = plan;
  gu.El = El;
  W4Args dn{};
  dn.A = h;
  dn.part = h_part;
  dn.codes = dn_codes;
  dn.scales = dn_scales;
  dn.K = F;
  dn.N = L.H;
  dn.w_rows = L.H;
  dn.Out = static_cast<bf16_t*>(out_buf);
  dn.out_perm = perm;
  dn.plan = plan;
  dn.El = El;
  if (bm == 32) {
    dn.split = tiling.parts;
    dn.split_stages = tiling.stages;
    dn.partial = reinterpret_cast<float*>(h + 2 * h_part);
    dn.partial_stride = rows * L.H;
  }
  const int64_t mtiles = ceil_div_host64(rows, bm) + El;
  if (bm == 32) launch_gemms<32, 1, 4, 2>(gu, dn, rows, mtiles, num_cus, stream);
  else if (bm == 128) launch_gemms<128, 2, 4, 1>(gu, dn, rows, mtiles, num_cus, stream);
  else launch_gemms<256, 2, 4, 1>(gu, dn, rows, mtiles, num_cus, stream);
  return hipGetLastError();
}

}  // namespace moe
