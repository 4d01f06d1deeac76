// Expert SwiGLU MLP on dispatched rows with 4-bit expert weights (moe_expert_mlp_w4).
//
// The plan (rows grouped by local expert, mlp.hip) and the two passes are moe_expert_mlp's: gate/up with
// h = silu(g) * u, then down. The weights are the M operand of the matrix unit (blocks of 16 output columns) and the
// rows its N operand, so a packed code tile, one contiguous kilobyte, is decoded in registers right into the
// operand it is (w4.h), and a lane ends up with four consecutive output columns of one row.
//
//   w4_stream_kernel  few rows per expert, bound by the bytes of the codes: every wave streams its own blocks'
//                     codes through registers, several K steps in flight; the rows' 128-k slices are shared through
//                     LDS (two buffers, one barrier per step).
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "mfma.h"
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
  int64_t out_part;      // elements from Out to the second part of h, 0: one rounding
  const int* out_perm;   // destination row of a plan row, or nullptr
  const int* plan;
  int El;
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// the last index i in [0, n) with first[i] * scale <= v (first ascending, first[0] = 0)
__device__ __forceinline__ int find_expert(const int* first, int n, int scale, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] * scale <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// This workgroup's tiles out of `total`: the list is cut into eight contiguous ranges, one per XCD (workgroup b runs
// on XCD b % 8), so tiles that share weights or rows meet in one L2.
struct Tiles {
  int begin, end, step;
};
__device__ __forceinline__ Tiles my_tiles(int total) {
  const int G = gridDim.x;
  Tiles t{(int)blockIdx.x, total, G};
  if ((G & 7) == 0) {
    const int x = blockIdx.x & 7, per = (total + 7) >> 3;
    t.begin = x * per + (blockIdx.x >> 3);
    t.end = min(total, (x + 1) * per);
    t.step = G >> 3;
  }
  return t;
}

// ------------------------------------------------------------------------------------------------
// few rows per expert
// ------------------------------------------------------------------------------------------------
// NB blocks of 16 rows; 8 waves, each two 16-row weight blocks: the gate and the up rows of the same 16 columns of h
// (a tile is 128 columns), or two neighbouring blocks of down rows (a tile is 256 columns). HP parts of the rows.
template <int NB, bool GATED, int HP>
__global__ __launch_bounds__(512) void w4_stream_kernel(W4Args a) {
  constexpr int NW = 8, BM = NB * 16, PF = 3;
  constexpr int COLS = GATED ? NW * 16 : NW * 32;
  constexpr int PITCH = 256 + 16;               // bytes of a staged row: 128 k and a vector of padding
  constexpr int XL = (BM * 16 + 511) / 512;     // 16-byte loads per thread, part and step
  __shared__ __attribute__((aligned(16))) unsigned char s_x[2][HP][BM * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = a.K, ns = (K + W4_TILE_K - 1) / W4_TILE_K, ks = (K + W4_STILE_K - 1) / W4_STILE_K;
  const int* row_start = a.plan + 2;
  const int* tile_start = a.plan + 3 + a.El;
  const int n_tiles = (a.N + COLS - 1) / COLS;
  const Tiles mine = my_tiles(a.plan[0] * n_tiles);
  for (int tile = mine.begin; tile < mine.end; tile += mine.step) {
    const int l = find_expert(tile_start, a.El, n_tiles, tile);
    const int mt_l = tile_start[l + 1] - tile_start[l];
    const int local = tile - tile_start[l] * n_tiles;
    const int nt = local / mt_l, mt = local % mt_l;
    const int p0 = row_start[l] + mt * BM, m_rows = min(BM, row_start[l + 1] - p0);
    // this wave's two weight blocks; blocks past N repeat the first one and are not stored
    const int c0 = nt * COLS + wave * (GATED ? 16 : 32);
    const bool on0 = c0 < a.N, on1 = GATED ? on0 : c0 + 16 < a.N;
    const int64_t base = (int64_t)l * a.w_rows;
    const int64_t b0 = (base + (on0 ? c0 : 0)) / 16;
    const int64_t b1 = GATED ? (base + a.up + (on0 ? c0 : 0)) / 16 : (base + (on1 ? c0 + 16 : 0)) / 16;
    const uint8_t* wc[2] = {a.codes + b0 * ns * W4_CODE_TILE + lane * 16, a.codes + b1 * ns * W4_CODE_TILE + lane * 16};
    const uint8_t* wsc[2] = {a.scales + b0 * ks * W4_SCALE_TILE + lane * 4, a.scales + b1 * ks * W4_SCALE_TILE + lane * 4};
    // this thread's rows of the shared slices: vector tid + i * 512 of BM x 16
    const bf16_t* src[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int r = min((tid + i * 512) >> 4, m_rows - 1);
      src[i] = a.A + (int64_t)(a.a_perm ? a.a_perm[p0 + r] : p0 + r) * K;
    }
    u32x4 rw[PF][2];
    uint32_t rs[PF][2];
    u32x4 rx[HP][XL];
    auto load_w = [&](int st, int u) {
      const int s = min(st, ns - 1);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        rw[u][b] = ld16_nt(wc[b] + (int64_t)s * W4_CODE_TILE);
        rs[u][b] = wsc[b][(s >> 2) * W4_SCALE_TILE + (s & 3)];
      }
    };
    auto load_x = [&](int st) {
      const int k = min(st, ns - 1) * W4_TILE_K + (tid & 15) * 8;
#pragma unroll
      for (int p = 0; p < HP; ++p)
#pragma unroll
        for (int i = 0; i < XL; ++i) rx[p][i] = ld16(src[i] + p * a.part + min(k, K - 8));
    };
    auto store_x = [&](int st) {
      const u32x4 zero = {0u, 0u, 0u, 0u};
      const bool in = st * W4_TILE_K + (tid & 15) * 8 < K;
#pragma unroll
      for (int p = 0; p < HP; ++p)
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          const int r = (tid + i * 512) >> 4;
          if (BM * 16 % 512 == 0 || r < BM) st16(s_x[st & 1][p] + r * PITCH + (tid & 15) * 16, in ? rx[p][i] : zero);
        }
    };
    f32x4 acc[2][NB];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[b][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    load_x(0);
#pragma unroll
    for (int u = 0; u < PF; ++u) load_w(u, u);
    store_x(0);
    load_x(1);
    lds_barrier();
    for (int s0 = 0; s0 < ns; s0 += PF) {
#pragma unroll
      for (int u = 0; u < PF; ++u) {
        const int st = s0 + u;
        if (st < ns) {
          const float sc0 = w4_scale(rs[u][0]), sc1 = w4_scale(rs[u][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4 f0[1] = {w4_to_bf16(rw[u][0][j], sc0)}, f1[1] = {w4_to_bf16(rw[u][1][j], sc1)};
#pragma unroll
            for (int p = 0; p < HP; ++p)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const u32x4 b[1] = {ld16(s_x[st & 1][p] + (nb * 16 + (lane & 15)) * PITCH + (lane >> 4) * 64 + j * 16)};
                Op16::step(acc[0][nb], f0, b);
                Op16::step(acc[1][nb], f1, b);
              }
          }
          load_w(st + PF, u);
          if (st + 1 < ns) {
            store_x(st + 1);
            load_x(st + 2);
          }
          lds_barrier();
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 16 + (lane & 15);
      if (r < m_rows) {
        const int64_t orow = a.out_perm ? a.out_perm[p0 + r] : p0 + r;
        const int q0 = (lane >> 4) * 4;
        if constexpr (GATED) {
          if (on0) {
            float h[4], rest[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              h[q] = silu(acc[0][nb][q]) * acc[1][nb][q];
              rest[q] = h[q] - (float)(bf16_t)h[q];
            }
            bf16_t* o = a.Out + orow * a.N + c0 + q0;
            *reinterpret_cast<u32x2*>(o) = u32x2{pack2_bf16(h[0], h[1]), pack2_bf16(h[2], h[3])};
            if (a.out_part != 0)
              *reinterpret_cast<u32x2*>(o + a.out_part) = u32x2{pack2_bf16(rest[0], rest[1]), pack2_bf16(rest[2], rest[3])};
          }
        } else {
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if (b ? on1 : on0)
              *reinterpret_cast<u32x2*>(a.Out + orow * a.N + c0 + b * 16 + q0) =
                  u32x2{pack2_bf16(acc[b][nb][0], acc[b][nb][1]), pack2_bf16(acc[b][nb][2], acc[b][nb][3])};
        }
      }
    }
  }
}

int w4_grid(int64_t tiles, int64_t most) {
  int64_t g = std::min(tiles, most);
  if (g >= 8) g &= ~7ll;
  return (int)std::max<int64_t>(g, 1);
}

template <int NB>
void launch_stream(const W4Args& gu, const W4Args& dn, int64_t mtiles, int num_cus, hipStream_t stream) {
  w4_stream_kernel<NB, true, 1><<<w4_grid(mtiles * ceil_div_host(gu.N, 128), 2 * num_cus), 512, 0, stream>>>(gu);
  w4_stream_kernel<NB, false, 2><<<w4_grid(mtiles * ceil_div_host(dn.N, 256), 2 * num_cus), 512, 0, stream>>>(dn);
}

// rows per M tile: the capacity per local expert bounds its rows
int w4_rows(int64_t rows_max, int El) {
  const int64_t per = El > 0 ? ceil_div_host64(rows_max, El) : rows_max;
  return per <= 16 ? 16 : per <= 32 ? 32 : 64;
}

}  // namespace

size_t mlp_w4_workspace_bytes(int64_t rows, int El, int F) {
  return align256(mlp_plan_ints(El) * sizeof(int)) + align256((size_t)rows * sizeof(int)) +
         2 * align256((size_t)rows * (size_t)F * 2);
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
  const int bm = w4_rows(rows, El);
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
  const int64_t mtiles = ceil_div_host64(rows, bm) + El;
  if (bm == 16) launch_stream<1>(gu, dn, mtiles, num_cus, stream);
  else if (bm == 32) launch_stream<2>(gu, dn, mtiles, num_cus, stream);
  else launch_stream<4>(gu, dn, mtiles, num_cus, stream);
  return hipGetLastError();
}

}  // namespace moe
