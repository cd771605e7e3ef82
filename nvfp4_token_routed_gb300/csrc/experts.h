// experts.h -- declarations shared by the kernels of the differentiable pass through
// routed experts (routes, activations kept in 8 bits, microscaled FP4) and their entry
// points.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "loss.h"  // the element types kF32, kBf16, kF16

namespace moe {

constexpr int kMxPanel = 256;  // values of a row per scale panel, and per GEMM stage

// ---------------------------------------------------------------- routes (routes.cu)
struct SortArgs {
  int T, K, E, ids64;
  const void* ids;   // int32 or int64 [T][K]
  int32_t* offsets;  // [E + 1]
  int32_t* perm;     // [T*K]
  int32_t* inv;      // [T][K]
  int32_t* status;   // kStatusWords words at the workspace's start, or null (one cluster)
  int32_t* chunks;   // [chunks][E + 1] then totals [E]
};
constexpr size_t kSortStatusBytes = 256;  // head of the workspace, all of it up to 32768 routes
size_t sort_routes_ws_bytes(int64_t TK, int E);
cudaError_t launch_sort_routes(const SortArgs& a, cudaStream_t s);

// Rows of T tokens and of their T*K routes.  Strides are in elements.
struct RowArgs {
  int T, K, H;
  const int32_t* inv;  // [T][K]; outside [0, T*K): an empty slot
  const void* x;       // dispatch: tokens; combine, its gradient: the routes' rows, or null
  int64_t ld_x;
  const float* w;      // [T][K], or null: 1
  const void* dout;    // combine's gradient: [T][H]
  int64_t ld_dout;
  void* out;           // dispatch, combine's gradient: the routes' rows; combine: [T][H]
  int64_t ld_out;
  float* dw;           // combine's gradient: [T][K], or null
};
cudaError_t launch_dispatch(const RowArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_combine(const RowArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_combine_grad(const RowArgs& a, int dtype, cudaStream_t s);
// A microscaled matrix of T rows of H values (a multiple of kMxPanel): codes in x and out.
cudaError_t launch_dispatch_mx(const RowArgs& a, const uint8_t* scales, uint8_t* out_scales,
                               cudaStream_t s);

// ---------------------------------------------------------------- 8 bits (checkpoint.cu)
struct KeepArgs {
  int R, W;              // rows; values a row and half
  const int32_t* n_rows; // device: rows that count (at most R), or null: R
  const void* x;         // checkpoint, act: input rows; act gradient: dy
  int64_t ld_x;
  uint8_t* codes;        // [R][halves][Wp], Wp = W rounded up to 32
  uint8_t* scales;       // [R][halves][Wp / 32]
  void* out;             // restore: rows; act: y; act gradient: dh
  int64_t ld_out;
  float limit;           // SwiGLU: > 0 clamped
};
enum KeepAct { kActRelu2 = 0, kActSwiglu = 1 };
cudaError_t launch_checkpoint(const KeepArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_restore(const KeepArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_expert_act(const KeepArgs& a, int act, int dtype, cudaStream_t s);
cudaError_t launch_expert_act_grad(const KeepArgs& a, int act, int dtype, cudaStream_t s);

// ---------------------------------------------------------------- microscaled FP4 (mx_quant.cu)
struct MxQuantArgs {
  int R, D, Dp;          // Dp = D rounded up to kMxPanel
  const int32_t* n_rows; // as KeepArgs
  const void* x;         // rows, or restored rows
  int64_t ld_x;
  uint8_t* codes;        // [R][Dp / 2]
  uint8_t* scales;       // [Dp / 256][Rp][8], Rp = R rounded up to 2
  void* out;             // restore
  int64_t ld_out;
};
cudaError_t launch_mx_quantize(const MxQuantArgs& a, int dtype, cudaStream_t s);
// x is a stack of [D][C] matrices (contiguous): row (b, c) of the result is column c of
// matrix b.  R = batch * C.
cudaError_t launch_mx_quantize_t(const MxQuantArgs& a, int C, int dtype, cudaStream_t s);
cudaError_t launch_mx_restore(const MxQuantArgs& a, int dtype, cudaStream_t s);

// ---------------------------------------------------------------- its product (gemm_mx.cu)
struct MxGemmArgs {
  int R, E, N, kblocks;    // rows, experts, outputs, Dp / 256
  const int32_t* offsets;  // [E + 1] device, or null: one group of all rows
  const uint8_t* sx;       // scale panels of the rows
  int64_t sx_panel;        // bytes a panel: 8 * Rp
  const uint8_t* sw;       // scale panels of the weights (E*N rows)
  int64_t sw_panel;
  void* out;               // [R][N], row stride ld
  int64_t ld;
  int dtype;
  int wide;                // 16-bit out in runs of 4 on 8 bytes
  int tile_rows;           // pairs: rows of the largest tile
  int leave_item;          // self-test: the token producer leaves before this item; -1: never
};
cudaError_t launch_gemm_mx(const MxGemmArgs& a, const uint8_t* x_codes, const uint8_t* w_codes,
                           int sms, cudaStream_t s);

}  // namespace moe
