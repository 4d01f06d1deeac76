// C ABI of the MoE-layer hot path: argument validation on the host, workspace carving, launches.
// Every entry point validates before its first HIP call, allocates nothing and only enqueues work on
// the caller's stream.
#include <string.h>

#include <mutex>

#include "common.h"
#include "kernels.h"

namespace {

// Scratch of moe_dispatch_noalloc: one static device array per GPU (each device that loads the library
// holds its own copy). In host code `scratch` names a host-side stand-in, not device memory: kernels and
// copies are only ever given the device address that hipGetSymbolAddress returns for the current device.
__device__ __align__(256) unsigned char scratch[MOE_DISPATCH_NOALLOC_MAX_WORKSPACE];
constexpr int kScratchDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kScratchDevices] = {};

// The device address of `scratch` on the current device, looked up on the first call there.
int scratch_address(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MOE_ERR_HIP;
  if (dev >= kScratchDevices) return MOE_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return MOE_ERR_HIP;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

// Compute units of the current device (cached per device id; a benign race fills the same value).
int device_cus() {
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
  if (dev < 64) cache[dev] = n;
  return n;
}

// the split-K plan of the router is fixed for the target chip (256 CUs), so the workspace size is a
// function of the shape alone
constexpr int ROUTE_PLAN_CUS = 256;

bool valid_dtype(moe_dtype_t d) { return d == MOE_F32 || d == MOE_BF16; }

// the kernels move activations, weights and rows in 16-byte vectors and int / fp32 arrays in 4-byte words
// (a null pointer passes: the null checks come first)
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_layout(const moe_layout_t* L) {
  if (!L) return MOE_ERR_INVALID;
  if (L->T < 0 || L->C < 0 || L->E < 1 || L->R < 1 || L->k < 1 || L->H < 1) return MOE_ERR_INVALID;
  if (L->E > MOE_MAX_EXPERTS || L->k > MOE_MAX_TOPK || L->k > L->E) return MOE_ERR_INVALID;
  if (L->E % L->R != 0) return MOE_ERR_INVALID;
  if (L->H % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)L->T * L->k > (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (!L->expert_count || !L->expert_kept || !L->expert_overflow || !L->expert_offset) return MOE_ERR_INVALID;
  const int64_t rows = moe_rows_max(L->T, L->k, L->E, L->C);
  if (rows > 0 && (!L->row_token || !L->row_slot)) return MOE_ERR_INVALID;
  if (L->T > 0 && !L->pair_row) return MOE_ERR_INVALID;
  if (!al4(L->expert_count) || !al4(L->expert_kept) || !al4(L->expert_overflow) || !al4(L->expert_offset) ||
      !al4(L->row_token) || !al4(L->row_slot) || !al4(L->pair_row))
    return MOE_ERR_INVALID;
  return MOE_OK;
}

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace

extern "C" {

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case MOE_ERR_HIP: return "HIP launch error";
    default: return "unknown status";
  }
}

int64_t moe_rows_max(int T, int k, int E, int C) {
  if (T <= 0 || k <= 0 || E <= 0 || C <= 0) return 0;
  const int64_t a = (int64_t)T * k, b = (int64_t)E * C;
  return a < b ? a : b;
}

size_t moe_route_workspace_bytes(int T, int H, int E, moe_dtype_t xdt) {
  if (T <= 0 || H <= 0 || E <= 0 || !valid_dtype(xdt)) return 0;
  const moe::RoutePlan plan = moe::route_plan(T, H, E, xdt == MOE_BF16, ROUTE_PLAN_CUS);
  return plan.planes_bytes + plan.partial_bytes;
}

int moe_route(const void* x, moe_dtype_t xdt, const float* w_router, const float* logit_bias,
              int64_t bias_row_stride, int T, int H, int E, int k, float* logits, int32_t* topk_ids,
              float* topk_w, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > MOE_MAX_TOPK || k > E)
    return MOE_ERR_INVALID;
  if (H % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (logit_bias && bias_row_stride < 0) return MOE_ERR_INVALID;
  if ((int64_t)T * E > (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !logits || !topk_ids || !topk_w) return MOE_ERR_INVALID;
  if (!al16(x) || !al16(w_router) || !al16(workspace) || !al4(logit_bias) || !al4(logits) || !al4(topk_ids) ||
      !al4(topk_w))
    return MOE_ERR_INVALID;
  const size_t need = moe_route_workspace_bytes(T, H, E, xdt);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID;
  const moe::RoutePlan plan = moe::route_plan(T, H, E, xdt == MOE_BF16, ROUTE_PLAN_CUS);
  return hip_status(moe::launch_route(x, xdt == MOE_BF16, w_router, logit_bias, logit_bias ? bias_row_stride : 0,
                                      T, H, E, k, logits, topk_ids, topk_w, workspace, plan, stream));
}

size_t moe_dispatch_workspace_bytes(int T, int k, int E) {
  if (T < 0 || k < 0 || E < 0) return 0;
  const size_t nblk = (size_t)moe::dispatch_num_blocks(T);
  return moe::align256(nblk * (size_t)E * sizeof(int)) + moe::align256((size_t)T * k * sizeof(int));
}

int moe_dispatch(const void* x, moe_dtype_t xdt, const int32_t* topk_ids, const moe_layout_t* layout,
                 void* send_buf, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (L.T > 0 && (!x || !topk_ids)) return MOE_ERR_INVALID;
  if (rows > 0 && !send_buf) return MOE_ERR_INVALID;
  if (!al16(x) || !al16(send_buf) || !al16(workspace) || !al4(topk_ids)) return MOE_ERR_INVALID;
  const size_t need = moe_dispatch_workspace_bytes(L.T, L.k, L.E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  int* blk_count = reinterpret_cast<int*>(ws);
  int* pair_local =
      reinterpret_cast<int*>(ws + moe::align256((size_t)moe::dispatch_num_blocks(L.T) * L.E * sizeof(int)));
  return hip_status(moe::launch_dispatch(x, xdt == MOE_BF16, topk_ids, L, send_buf, blk_count, pair_local, stream));
}

int moe_dispatch_noalloc(const void* x, moe_dtype_t xdt, const int32_t* topk_ids, const moe_layout_t* layout,
                         void* send_buf, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (L.T > 0 && (!x || !topk_ids)) return MOE_ERR_INVALID;
  if (rows > 0 && !send_buf) return MOE_ERR_INVALID;
  if (!al16(x) || !al16(send_buf) || !al4(topk_ids)) return MOE_ERR_INVALID;
  if (moe_dispatch_workspace_bytes(L.T, L.k, L.E) > MOE_DISPATCH_NOALLOC_MAX_WORKSPACE) return MOE_ERR_UNSUPPORTED;
  void* ws = nullptr;
  const int sst = scratch_address(&ws);
  if (sst != MOE_OK) return sst;
  // the same carving as moe_dispatch's workspace; the kernels write every entry they later read, so
  // the array's contents from an earlier call need no clearing
  char* base = static_cast<char*>(ws);
  int* blk_count = reinterpret_cast<int*>(base);
  int* pair_local =
      reinterpret_cast<int*>(base + moe::align256((size_t)moe::dispatch_num_blocks(L.T) * L.E * sizeof(int)));
  return hip_status(moe::launch_dispatch(x, xdt == MOE_BF16, topk_ids, L, send_buf, blk_count, pair_local, stream));
}

size_t moe_expert_mlp_workspace_bytes(int T, int k, int E, int R, int C, int F, moe_dtype_t xdt) {
  if (E <= 0 || R <= 0 || E % R != 0 || F <= 0) return 0;
  const int El = E / R;
  const int64_t rows = moe_rows_max(T, k, E, C);
  const size_t esz = xdt == MOE_BF16 ? 2 : 4;
  return moe::align256(moe::mlp_plan_ints(El) * sizeof(int)) + moe::align256((size_t)rows * sizeof(int)) +
         moe::align256((size_t)rows * (size_t)F * esz);
}

namespace {
// counters of the fused combine: one per (token, down-GEMM column band)
size_t combine_counter_bytes(int T, int k, int E, int R, int C, int H, int F, moe_dtype_t xdt) {
  const int64_t rows = moe_rows_max(T, k, E, C);
  const moe::MlpTiles tiles = moe::mlp_pick_tiles(rows, E / R, H, F, xdt == MOE_BF16);
  const int64_t bands = (H + moe::mlp_down_cols(tiles) - 1) / moe::mlp_down_cols(tiles);
  return moe::align256((size_t)((int64_t)T * bands) * sizeof(int));
}
}  // namespace

size_t moe_expert_mlp_combine_workspace_bytes(int T, int k, int E, int R, int C, int H, int F, moe_dtype_t xdt) {
  if (E <= 0 || R <= 0 || E % R != 0 || F <= 0 || H <= 0 || T < 0) return 0;
  return moe_expert_mlp_workspace_bytes(T, k, E, R, C, F, xdt) + combine_counter_bytes(T, k, E, R, C, H, F, xdt);
}

namespace {
// Shared by moe_expert_mlp, moe_expert_mlp_fp8 and moe_expert_mlp_combine: validation, workspace carving,
// launch. a_scale != nullptr means send_buf holds E4M3 codes with these block scales; y != nullptr fuses
// the combine into the down GEMM.
int expert_mlp(const void* send_buf, const float* a_scale, moe_dtype_t xdt, const moe_layout_t* layout,
               const void* w_gate_up, const void* w_down, int F, void* out_buf, void* workspace,
               size_t workspace_bytes, hipStream_t stream, const float* topk_w = nullptr, void* y = nullptr) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (F < 1) return MOE_ERR_INVALID;
  if (F % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)2 * F > (int64_t)INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (!w_gate_up || !w_down) return MOE_ERR_INVALID;
  if (rows > 0 && (!send_buf || !out_buf)) return MOE_ERR_INVALID;
  if (!al16(send_buf) || !al16(w_gate_up) || !al16(w_down) || !al16(out_buf) || !al16(workspace) || !al16(y) ||
      !al4(topk_w) || !al4(a_scale))
    return MOE_ERR_INVALID;
  const size_t need = y ? moe_expert_mlp_combine_workspace_bytes(L.T, L.k, L.E, L.R, L.C, L.H, F, xdt)
                        : moe_expert_mlp_workspace_bytes(L.T, L.k, L.E, L.R, L.C, F, xdt);
  if (!workspace || workspace_bytes < need) return MOE_ERR_INVALID;
  const int El = L.E / L.R;
  char* ws = static_cast<char*>(workspace);
  int* plan = reinterpret_cast<int*>(ws);
  ws += moe::align256(moe::mlp_plan_ints(El) * sizeof(int));
  int* perm = reinterpret_cast<int*>(ws);
  ws += moe::align256((size_t)rows * sizeof(int));
  void* hbuf = ws;
  ws += moe::align256((size_t)rows * (size_t)F * (xdt == MOE_BF16 ? 2 : 4));
  int* counter = y ? reinterpret_cast<int*>(ws) : nullptr;
  const moe::MlpTiles tiles = moe::mlp_pick_tiles(rows, El, L.H, F, xdt == MOE_BF16);
  return hip_status(moe::launch_expert_mlp(send_buf, xdt == MOE_BF16, L, w_gate_up, w_down, F, out_buf, plan, perm,
                                           hbuf, tiles, device_cus(), stream, a_scale, topk_w, y, counter));
}

}  // namespace

int moe_expert_mlp(const void* send_buf, moe_dtype_t xdt, const moe_layout_t* layout, const void* w_gate_up,
                   const void* w_down, int F, void* out_buf, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
  return expert_mlp(send_buf, nullptr, xdt, layout, w_gate_up, w_down, F, out_buf, workspace, workspace_bytes,
                    stream);
}

int moe_expert_mlp_combine(const void* send_buf, moe_dtype_t xdt, const moe_layout_t* layout, const void* w_gate_up,
                           const void* w_down, int F, const float* topk_w, void* out_buf, void* y, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  if (layout->T > 0 && (!topk_w || !y)) return MOE_ERR_INVALID;
  if (layout->T == 0) {  // nothing to combine: the plain expert MLP (its plan kernel only)
    return expert_mlp(send_buf, nullptr, xdt, layout, w_gate_up, w_down, F, out_buf, workspace, workspace_bytes,
                      stream);
  }
  return expert_mlp(send_buf, nullptr, xdt, layout, w_gate_up, w_down, F, out_buf, workspace, workspace_bytes,
                    stream, topk_w, y);
}

int moe_dispatch_fp8(const void* x, moe_dtype_t xdt, const int32_t* topk_ids, const moe_layout_t* layout,
                     uint8_t* send_q, float* send_scale, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
  if (xdt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (L.H % MOE_FP8_BLOCK != 0) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (L.T > 0 && (!x || !topk_ids)) return MOE_ERR_INVALID;
  if (rows > 0 && (!send_q || !send_scale)) return MOE_ERR_INVALID;
  if (!al16(x) || !al16(send_q) || !al16(workspace) || !al4(send_scale) || !al4(topk_ids)) return MOE_ERR_INVALID;
  const size_t need = moe_dispatch_workspace_bytes(L.T, L.k, L.E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  int* blk_count = reinterpret_cast<int*>(ws);
  int* pair_local =
      reinterpret_cast<int*>(ws + moe::align256((size_t)moe::dispatch_num_blocks(L.T) * L.E * sizeof(int)));
  return hip_status(moe::launch_dispatch_fp8(x, topk_ids, L, send_q, send_scale, blk_count, pair_local, stream));
}

int moe_expert_mlp_fp8(const uint8_t* send_q, const float* send_scale, const moe_layout_t* layout,
                       const void* w_gate_up, const void* w_down, int F, void* out_buf, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (L.H % MOE_FP8_BLOCK != 0) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (rows > 0 && !send_scale) return MOE_ERR_INVALID;
  // with no rows there is nothing to decode: the bf16 path launches only the (empty) plan
  return expert_mlp(send_q, rows > 0 ? send_scale : nullptr, MOE_BF16, layout, w_gate_up, w_down, F, out_buf,
                    workspace, workspace_bytes, stream);
}

int moe_combine(const void* out_buf, moe_dtype_t xdt, const moe_layout_t* layout, const float* topk_w, void* y,
                hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (L.T == 0) return MOE_OK;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (!topk_w || !y) return MOE_ERR_INVALID;
  if (rows > 0 && !out_buf) return MOE_ERR_INVALID;
  if (!al16(out_buf) || !al16(y) || !al4(topk_w)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_combine(out_buf, xdt == MOE_BF16, L, topk_w, y, stream));
}

int moe_combine_send(const void* out_buf, moe_dtype_t xdt, const moe_layout_t* layout, const float* topk_w,
                     void* partial, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (L.T == 0) return MOE_OK;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  if (!topk_w || !partial) return MOE_ERR_INVALID;
  if (rows > 0 && !out_buf) return MOE_ERR_INVALID;
  if (!al16(out_buf) || !al16(partial) || !al4(topk_w)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_combine_send(out_buf, xdt == MOE_BF16, L, topk_w, partial, stream));
}

int moe_combine_recv(const void* partial, moe_dtype_t xdt, const moe_layout_t* layout, void* y, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  if (L.T == 0) return MOE_OK;
  if (!partial || !y) return MOE_ERR_INVALID;
  if (!al16(partial) || !al16(y)) return MOE_ERR_INVALID;
  return hip_status(moe::launch_combine_recv(partial, xdt == MOE_BF16, L, y, stream));
}

namespace {
// sizes a packed matrix may have: whole groups and row blocks, and no more weights than bytes can be counted for
bool w4_sizes(int64_t rows, int K) {
  return rows % 16 == 0 && K % MOE_W4_GROUP == 0 && K <= INT32_MAX - 512 && rows <= INT64_MAX / 4 / K;
}
}  // namespace

size_t moe_w4_codes_bytes(int64_t rows, int K) {
  if (rows <= 0 || K <= 0 || !w4_sizes(rows, K)) return 0;
  return (size_t)(rows / 16) * (size_t)moe::ceil_div_host(K, 128) * 1024;
}

size_t moe_w4_scales_bytes(int64_t rows, int K) {
  if (rows <= 0 || K <= 0 || !w4_sizes(rows, K)) return 0;
  return (size_t)(rows / 16) * (size_t)moe::ceil_div_host(K, 512) * 256;
}

namespace {
// Shared by moe_quantize_w4 and moe_dequantize_w4
int check_w4(const void* w, moe_dtype_t wdt, int64_t rows, int K, const void* codes, const void* scales) {
  if (!valid_dtype(wdt)) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || K < 1) return MOE_ERR_INVALID;
  if (!w4_sizes(rows, K)) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!w || !codes || !scales)) return MOE_ERR_INVALID;
  if (!al16(w) || !al16(codes) || !al16(scales)) return MOE_ERR_INVALID;
  return MOE_OK;
}
}  // namespace

int moe_quantize_w4(const void* w, moe_dtype_t wdt, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                    hipStream_t stream) {
  const int st = check_w4(w, wdt, rows, K, codes, scales);
  if (st != MOE_OK || rows == 0) return st;
  return hip_status(moe::launch_quantize_w4(w, wdt == MOE_BF16, rows, K, codes, scales, stream));
}

int moe_dequantize_w4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, void* w, moe_dtype_t wdt,
                      hipStream_t stream) {
  const int st = check_w4(w, wdt, rows, K, codes, scales);
  if (st != MOE_OK || rows == 0) return st;
  return hip_status(moe::launch_dequantize_w4(codes, scales, rows, K, w, wdt == MOE_BF16, stream));
}

size_t moe_expert_mlp_w4_workspace_bytes(int T, int k, int E, int R, int C, int F) {
  if (E <= 0 || R <= 0 || E % R != 0 || F <= 0) return 0;
  const int64_t rows = moe_rows_max(T, k, E, C);
  if (rows > INT32_MAX || !moe::mlp_w4_fits(rows, MOE_W4_GROUP, F)) return 0;  // for no H
  return moe::mlp_w4_workspace_bytes(rows, E / R, F);
}

namespace {
// The widths moe_expert_mlp_w4 takes for `rows` rows
int check_w4_widths(int64_t rows, int H, int F) {
  if (F < 1) return MOE_ERR_INVALID;
  if (H % MOE_W4_GROUP != 0 || F % MOE_W4_GROUP != 0) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)2 * F > (int64_t)INT32_MAX / 2 || H > INT32_MAX / 4) return MOE_ERR_UNSUPPORTED;
  return moe::mlp_w4_fits(rows, H, F) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
}  // namespace

int moe_expert_mlp_w4_tiling(int T, int k, int E, int R, int C, int H, int F, int* tile_rows, int* down_parts) {
  if (T < 0 || C < 0 || E < 1 || E > MOE_MAX_EXPERTS || R < 1 || E % R != 0 || k < 1 || k > MOE_MAX_TOPK || k > E ||
      H < 1 || !tile_rows || !down_parts)
    return MOE_ERR_INVALID;
  if ((int64_t)T * k > (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = moe_rows_max(T, k, E, C);
  const int st = check_w4_widths(rows, H, F);
  if (st != MOE_OK) return st;
  const moe::W4Tiling t = moe::mlp_w4_tiling(rows, E / R, H, F, device_cus());
  *tile_rows = t.rows;
  *down_parts = t.parts;
  return MOE_OK;
}

int moe_expert_mlp_w4(const void* send_buf, const moe_layout_t* layout, const uint8_t* gu_codes,
                      const uint8_t* gu_scales, const uint8_t* dn_codes, const uint8_t* dn_scales, int F,
                      void* out_buf, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_layout(layout);
  if (st != MOE_OK) return st;
  const moe_layout_t& L = *layout;
  const int64_t rows = moe_rows_max(L.T, L.k, L.E, L.C);
  const int wst = check_w4_widths(rows, L.H, F);
  if (wst != MOE_OK) return wst;
  if (!gu_codes || !gu_scales || !dn_codes || !dn_scales) return MOE_ERR_INVALID;
  if (rows > 0 && (!send_buf || !out_buf)) return MOE_ERR_INVALID;
  if (!al16(send_buf) || !al16(gu_codes) || !al16(gu_scales) || !al16(dn_codes) || !al16(dn_scales) ||
      !al16(out_buf) || !al16(workspace))
    return MOE_ERR_INVALID;
  if (!workspace || workspace_bytes < moe_expert_mlp_w4_workspace_bytes(L.T, L.k, L.E, L.R, L.C, F))
    return MOE_ERR_INVALID;
  return hip_status(moe::launch_expert_mlp_w4(send_buf, L, gu_codes, gu_scales, dn_codes, dn_scales, F, out_buf,
                                              workspace, device_cus(), stream));
}

size_t moe_layer_decode_workspace_bytes(int T, int H, int E, int k, int F, moe_dtype_t xdt) {
  if (T <= 0 || T > MOE_DECODE_MAX_TOKENS || H <= 0 || E <= 0 || k <= 0 || k > MOE_MAX_TOPK || F <= 0 ||
      !valid_dtype(xdt) || H > moe::kDecodeMaxH || F > moe::kDecodeMaxF)
    return 0;
  return moe::decode_workspace_bytes(T, H, k, F);
}

namespace {
// Shared by moe_layer_decode and moe_layer_decode_w4 (packed): validation and launch. `unit` divides H and F.
int layer_decode(moe::DecodeCall& d, moe_dtype_t xdt, bool packed, size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(xdt)) return MOE_ERR_UNSUPPORTED;
  if (d.T < 0 || d.H < 1 || d.E < 1 || d.E > MOE_MAX_EXPERTS || d.R < 1 || d.E % d.R != 0 || d.k < 1 ||
      d.k > MOE_MAX_TOPK || d.k > d.E || d.C < 0 || d.F < 1)
    return MOE_ERR_INVALID;
  const int unit = packed ? MOE_W4_GROUP : 8;
  if (d.T > MOE_DECODE_MAX_TOKENS || d.H % unit != 0 || d.F % unit != 0) return MOE_ERR_UNSUPPORTED;
  // x, and h of one expert's rows in its two parts, are read at 31-bit byte offsets
  if (d.H > moe::kDecodeMaxH || d.F > moe::kDecodeMaxF) return MOE_ERR_UNSUPPORTED;
  if (d.bias && d.bias_stride < 0) return MOE_ERR_INVALID;
  if (d.T == 0) return MOE_OK;
  if (!d.x || !d.w_router || !d.w_gu || !d.w_dn || (packed && (!d.s_gu || !d.s_dn)) || !d.logits || !d.ids || !d.wts ||
      !d.y)
    return MOE_ERR_INVALID;
  if (!al16(d.x) || !al16(d.w_router) || !al16(d.w_gu) || !al16(d.w_dn) || !al16(d.s_gu) || !al16(d.s_dn) ||
      !al16(d.y) || !al16(d.workspace) || !al4(d.bias) || !al4(d.logits) || !al4(d.ids) || !al4(d.wts))
    return MOE_ERR_INVALID;
  if (!d.workspace || workspace_bytes < moe_layer_decode_workspace_bytes(d.T, d.H, d.E, d.k, d.F, xdt))
    return MOE_ERR_INVALID;
  d.bf16 = xdt == MOE_BF16;
  if (!d.bias) d.bias_stride = 0;
  return hip_status(moe::launch_layer_decode(d, device_cus(), stream));
}
}  // namespace

int moe_layer_decode(const void* x, moe_dtype_t xdt, const float* w_router, const float* logit_bias,
                     int64_t bias_row_stride, int T, int H, int E, int R, int k, int C, int F,
                     const void* w_gate_up, const void* w_down, float* logits, int32_t* topk_ids, float* topk_w,
                     void* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe::DecodeCall d{x,      0, w_router, logit_bias, bias_row_stride, T,        H,      E, R,        k, C, F, w_gate_up,
                    w_down, nullptr, nullptr, logits, topk_ids, topk_w, y, workspace};
  return layer_decode(d, xdt, false, workspace_bytes, stream);
}

int moe_layer_decode_w4(const void* x, const float* w_router, const float* logit_bias, int64_t bias_row_stride,
                        int T, int H, int E, int R, int k, int C, int F, const uint8_t* gu_codes,
                        const uint8_t* gu_scales, const uint8_t* dn_codes, const uint8_t* dn_scales, float* logits,
                        int32_t* topk_ids, float* topk_w, void* y, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  moe::DecodeCall d{x,        0,         w_router,  logit_bias, bias_row_stride, T,        H,      E, R, k, C, F, gu_codes,
                    dn_codes, gu_scales, dn_scales, logits,     topk_ids,        topk_w, y, workspace};
  return layer_decode(d, MOE_BF16, true, workspace_bytes, stream);
}

}  // extern "C"
