// experts_api.cu -- entry points of the differentiable pass through routed experts:
// argument checks and the launch.  No allocation and no host synchronisation.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_nvfp4.h"
#include "experts.h"
#include "internal.h"

using namespace moe;

namespace {

constexpr int64_t kMaxRoutes = int64_t(1) << 26;
constexpr int kMaxHidden = 65536;
constexpr int kMaxKept = 1 << 20;  // values of a kept row

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
uintptr_t dtype_size(int32_t d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
bool bool_ok(int32_t b) { return b == 0 || b == 1; }
moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // reported here, not by the next call
  return MOE_ERR_CUDA;
}
cudaStream_t raw(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Shape of a matrix of rows; its pointer is checked by check_ptr where it has rows.
moe_status check_rows(const moe_rows* x, int64_t max_rows, int32_t max_cols) {
  if (!x || x->rows < 0 || x->cols < 1 || !dtype_ok(x->dtype) || x->ld < x->cols)
    return MOE_ERR_INVALID_ARG;
  return x->rows > max_rows || x->cols > max_cols ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}
moe_status check_ptr(const void* p, int32_t dtype) {
  if (!p) return MOE_ERR_INVALID_ARG;
  return aligned(p, dtype_size(dtype)) ? MOE_OK : MOE_ERR_MISALIGNED;
}

moe_status check_routes(int32_t T, int32_t K) {
  if (T < 0 || K < 1) return MOE_ERR_INVALID_ARG;
  return K > 32 || (int64_t)T * K > kMaxRoutes ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

moe_status check_mx(const moe_mx* m) {
  if (!m || m->rows < 0 || m->cols < 1) return MOE_ERR_INVALID_ARG;
  if (m->rows > kMaxRoutes || m->cols > kMaxHidden) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (m->rows == 0) return MOE_OK;
  if (!m->codes || !m->scales) return MOE_ERR_INVALID_ARG;
  return aligned(m->codes, 16) && aligned(m->scales, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}
int padded(int32_t D) { return (D + kMxPanel - 1) / kMxPanel * kMxPanel; }

KeepArgs keep_args(int R, int W, const void* x, int64_t ld_x, const uint8_t* codes,
                   const uint8_t* scales, void* out, int64_t ld_out, float limit,
                   const int32_t* n_rows) {
  KeepArgs a = {};
  a.R = R;
  a.W = W;
  a.n_rows = n_rows;
  a.x = x;
  a.ld_x = ld_x;
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.out = out;
  a.ld_out = ld_out;
  a.limit = limit;
  return a;
}

MxQuantArgs quant_args(const moe_mx* m, const moe_rows* x, const int32_t* n_rows) {
  MxQuantArgs a = {};
  a.R = m->rows;
  a.D = m->cols;
  a.Dp = padded(m->cols);
  a.n_rows = n_rows;
  a.codes = m->codes;
  a.scales = m->scales;
  a.x = x ? x->data : nullptr;
  a.ld_x = x ? x->ld : 0;
  return a;
}

moe_status check_act(int32_t act, float limit) {
  if (act != MOE_ACT_RELU2 && act != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (!(limit >= 0.0f) || limit > 3.0e38f || (limit > 0.0f && act != MOE_ACT_SWIGLU))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status product_impl(const moe_mx* x, const moe_mx* w, int32_t E, const int32_t* offsets,
                        int32_t dtype, void* out, int64_t ld_out, int32_t leave,
                        moe_stream_t stream) {
  moe_status st = check_mx(x);
  if (st != MOE_OK || (st = check_mx(w)) != MOE_OK) return st;
  if (E < 1 || !dtype_ok(dtype) || w->rows < 1 || x->cols != w->cols || w->rows % E != 0 ||
      (!offsets && E != 1))
    return MOE_ERR_INVALID_ARG;
  const int N = w->rows / E;
  if (E > 1024 || N > kMaxHidden) return MOE_ERR_UNSUPPORTED_SHAPE;
  // offsets that do not ascend may put all rows into each of the groups: the kernels count
  // their tiles in 32 bits
  if (((int64_t)x->rows + 191) / 192 * ((N + 127) / 128) * E > INT32_MAX)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ld_out < N) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if ((st = check_ptr(out, dtype)) != MOE_OK) return st;
  if (!aligned(offsets, 4)) return MOE_ERR_MISALIGNED;
  int sms = 0;
  if ((st = (moe_status)device_status(&sms)) != MOE_OK) return st;
  MxGemmArgs a = {};
  a.R = x->rows;
  a.E = E;
  a.N = N;
  a.kblocks = padded(x->cols) / kMxPanel;
  a.offsets = offsets;
  a.sx = x->scales;
  a.sx_panel = 8 * (((int64_t)x->rows + 1) & ~int64_t(1));
  a.sw = w->scales;
  a.sw_panel = 8 * (((int64_t)w->rows + 1) & ~int64_t(1));
  a.out = out;
  a.ld = ld_out;
  a.dtype = dtype;
  a.wide = N % 4 == 0 && ld_out % 4 == 0 && aligned(out, 8);
  a.leave_item = leave;
  return cuda_status(launch_gemm_mx(a, x->codes, w->codes, sms, raw(stream)));
}

}  // namespace

extern "C" {

size_t moe_nvfp4_sort_routes_workspace_bytes(int32_t T, int32_t K, int32_t E) {
  if (check_routes(T, K) != MOE_OK || E < 1 || E > 1024 || K > E) return 0;
  return sort_routes_ws_bytes((int64_t)T * K, E);
}

moe_status moe_nvfp4_sort_routes(int32_t T, int32_t K, int32_t E, const void* topk_ids,
                                 int32_t ids_int64, int32_t* offsets, int32_t* perm, int32_t* inv,
                                 void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_routes(T, K);
  if (st != MOE_OK) return st;
  if (E < 1 || !bool_ok(ids_int64)) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || K > E) return MOE_ERR_UNSUPPORTED_SHAPE;
  const size_t need = sort_routes_ws_bytes((int64_t)T * K, E);
  if (!offsets || (!ws && need > kSortStatusBytes) || (T > 0 && (!topk_ids || !perm || !inv)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(ws, 256) || !aligned(perm, 4) || !aligned(inv, 4) ||
      (T > 0 && !aligned(topk_ids, ids_int64 ? 8 : 4)))
    return MOE_ERR_MISALIGNED;
  if (ws && ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(offsets, 0, ((size_t)E + 1) * sizeof(int32_t), raw(stream));
    if (e == cudaSuccess && ws)
      e = cudaMemsetAsync(ws, 0, kStatusWords * sizeof(int32_t), raw(stream));
    return cuda_status(e);
  }
  SortArgs a = {};
  a.T = T;
  a.K = K;
  a.E = E;
  a.ids = topk_ids;
  a.ids64 = ids_int64;
  a.offsets = offsets;
  a.perm = perm;
  a.inv = inv;
  a.status = static_cast<int32_t*>(ws);
  a.chunks = ws ? static_cast<int32_t*>(ws) + kSortStatusBytes / sizeof(int32_t) : nullptr;
  return cuda_status(launch_sort_routes(a, raw(stream)));
}

moe_status moe_nvfp4_dispatch(const moe_rows* x, int32_t K, const int32_t* inv, void* rows,
                              int64_t ld_rows, moe_stream_t stream) {
  moe_status st = check_rows(x, kMaxRoutes, kMaxHidden);
  if (st != MOE_OK || (st = check_routes(x->rows, K)) != MOE_OK) return st;
  if (ld_rows < x->cols) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if (!inv) return MOE_ERR_INVALID_ARG;
  if ((st = check_ptr(x->data, x->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(rows, x->dtype)) != MOE_OK) return st;
  if (!aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  RowArgs a = {};
  a.T = x->rows;
  a.K = K;
  a.H = x->cols;
  a.inv = inv;
  a.x = x->data;
  a.ld_x = x->ld;
  a.out = rows;
  a.ld_out = ld_rows;
  return cuda_status(launch_dispatch(a, x->dtype, raw(stream)));
}

moe_status moe_nvfp4_combine(const moe_rows* rows, int32_t T, int32_t K, const int32_t* inv,
                             const float* topk_w, void* out, int64_t ld_out,
                             moe_stream_t stream) {
  moe_status st = check_rows(rows, kMaxRoutes, kMaxHidden);
  if (st != MOE_OK || (st = check_routes(T, K)) != MOE_OK) return st;
  if (rows->rows != (int64_t)T * K || ld_out < rows->cols) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!inv) return MOE_ERR_INVALID_ARG;
  if ((st = check_ptr(rows->data, rows->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(out, rows->dtype)) != MOE_OK) return st;
  if (!aligned(inv, 4) || !aligned(topk_w, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  RowArgs a = {};
  a.T = T;
  a.K = K;
  a.H = rows->cols;
  a.inv = inv;
  a.x = rows->data;
  a.ld_x = rows->ld;
  a.w = topk_w;
  a.out = out;
  a.ld_out = ld_out;
  return cuda_status(launch_combine(a, rows->dtype, raw(stream)));
}

moe_status moe_nvfp4_combine_grad(const moe_rows* rows, int32_t T, int32_t K, const int32_t* inv,
                                  const float* topk_w, const void* dout, int64_t ld_dout,
                                  void* drows, int64_t ld_drows, float* d_topk_w,
                                  moe_stream_t stream) {
  moe_status st = check_rows(rows, kMaxRoutes, kMaxHidden);
  if (st != MOE_OK || (st = check_routes(T, K)) != MOE_OK) return st;
  if (rows->rows != (int64_t)T * K || ld_dout < rows->cols || ld_drows < rows->cols)
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!inv) return MOE_ERR_INVALID_ARG;
  if (d_topk_w && (st = check_ptr(rows->data, rows->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(dout, rows->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(drows, rows->dtype)) != MOE_OK) return st;
  if (!aligned(inv, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  RowArgs a = {};
  a.T = T;
  a.K = K;
  a.H = rows->cols;
  a.inv = inv;
  a.x = d_topk_w ? rows->data : nullptr;
  a.ld_x = rows->ld;
  a.w = topk_w;
  a.dout = dout;
  a.ld_dout = ld_dout;
  a.out = drows;
  a.ld_out = ld_drows;
  a.dw = d_topk_w;
  return cuda_status(launch_combine_grad(a, rows->dtype, raw(stream)));
}

moe_status moe_nvfp4_checkpoint(const moe_rows* x, uint8_t* codes, uint8_t* scales,
                                const int32_t* n_rows, moe_stream_t stream) {
  moe_status st = check_rows(x, kMaxRoutes, kMaxKept);
  if (st != MOE_OK || x->rows == 0) return st;
  if ((st = check_ptr(x->data, x->dtype)) != MOE_OK) return st;
  if (!codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 8) || !aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  return cuda_status(launch_checkpoint(
      keep_args(x->rows, x->cols, x->data, x->ld, codes, scales, nullptr, 0, 0.0f, n_rows),
      x->dtype, raw(stream)));
}

moe_status moe_nvfp4_restore(const uint8_t* codes, const uint8_t* scales, const moe_rows* out,
                             const int32_t* n_rows, moe_stream_t stream) {
  moe_status st = check_rows(out, kMaxRoutes, kMaxKept);
  if (st != MOE_OK || out->rows == 0) return st;
  if ((st = check_ptr(out->data, out->dtype)) != MOE_OK) return st;
  if (!codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 8) || !aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  return cuda_status(launch_restore(keep_args(out->rows, out->cols, nullptr, 0, codes, scales,
                                              const_cast<void*>(out->data), out->ld, 0.0f, n_rows),
                                    out->dtype, raw(stream)));
}

moe_status moe_nvfp4_expert_act(const moe_rows* h, int32_t act, float swiglu_limit, void* y,
                                int64_t ld_y, uint8_t* codes, uint8_t* scales,
                                const int32_t* n_rows, moe_stream_t stream) {
  moe_status st = check_act(act, swiglu_limit);
  if (st != MOE_OK || (st = check_rows(h, kMaxRoutes, kMaxKept)) != MOE_OK) return st;
  const int halves = act == MOE_ACT_SWIGLU ? 2 : 1;
  if (h->cols % halves != 0 || ld_y < h->cols / halves || !codes != !scales)
    return MOE_ERR_INVALID_ARG;
  const int I = h->cols / halves;
  if (I > kMaxKept / 2) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (h->rows == 0) return MOE_OK;
  if ((st = check_ptr(h->data, h->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(y, h->dtype)) != MOE_OK) return st;
  if (!aligned(codes, 8) || !aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  return cuda_status(launch_expert_act(
      keep_args(h->rows, I, h->data, h->ld, codes, scales, y, ld_y, swiglu_limit, n_rows), act,
      h->dtype, raw(stream)));
}

moe_status moe_nvfp4_expert_act_grad(const uint8_t* codes, const uint8_t* scales, int32_t act,
                                     float swiglu_limit, const moe_rows* dy, void* dh,
                                     int64_t ld_dh, const int32_t* n_rows, moe_stream_t stream) {
  moe_status st = check_act(act, swiglu_limit);
  if (st != MOE_OK || (st = check_rows(dy, kMaxRoutes, kMaxKept / 2)) != MOE_OK) return st;
  const int halves = act == MOE_ACT_SWIGLU ? 2 : 1;
  if (ld_dh < (int64_t)dy->cols * halves) return MOE_ERR_INVALID_ARG;
  if (dy->rows == 0) return MOE_OK;
  if ((st = check_ptr(dy->data, dy->dtype)) != MOE_OK) return st;
  if ((st = check_ptr(dh, dy->dtype)) != MOE_OK) return st;
  if (!codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 8) || !aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  return cuda_status(launch_expert_act_grad(
      keep_args(dy->rows, dy->cols, dy->data, dy->ld, codes, scales, dh, ld_dh, swiglu_limit,
                n_rows),
      act, dy->dtype, raw(stream)));
}

moe_status moe_nvfp4_mx_sizes(int32_t rows, int32_t cols, size_t bytes_out[2]) {
  if (rows < 0 || cols < 1 || !bytes_out) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRoutes || cols > kMaxHidden) return MOE_ERR_UNSUPPORTED_SHAPE;
  bytes_out[0] = (size_t)rows * (padded(cols) / 2);
  bytes_out[1] = (((size_t)rows + 1) & ~size_t(1)) * (padded(cols) / 32);
  return MOE_OK;
}

moe_status moe_nvfp4_mx_quantize(const moe_rows* x, const moe_mx* out, const int32_t* n_rows,
                                 moe_stream_t stream) {
  moe_status st = check_rows(x, kMaxRoutes, kMaxHidden);
  if (st != MOE_OK || (st = check_mx(out)) != MOE_OK) return st;
  if (x->rows != out->rows || x->cols != out->cols) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if ((st = check_ptr(x->data, x->dtype)) != MOE_OK) return st;
  if (!aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  return cuda_status(launch_mx_quantize(quant_args(out, x, n_rows), x->dtype, raw(stream)));
}

moe_status moe_nvfp4_mx_quantize_transposed(int32_t batch, int32_t D, int32_t C, const void* x,
                                            int32_t dtype, const moe_mx* out,
                                            moe_stream_t stream) {
  moe_status st = check_mx(out);
  if (st != MOE_OK) return st;
  if (batch < 0 || D < 1 || C < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (batch > 1024 || C > kMaxHidden) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (out->rows != (int64_t)batch * C || out->cols != D) return MOE_ERR_INVALID_ARG;
  if (batch == 0) return MOE_OK;
  if ((st = check_ptr(x, dtype)) != MOE_OK) return st;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  MxQuantArgs a = quant_args(out, nullptr, nullptr);
  a.x = x;
  return cuda_status(launch_mx_quantize_t(a, C, dtype, raw(stream)));
}

moe_status moe_nvfp4_mx_restore(const moe_mx* x, const moe_rows* out, const int32_t* n_rows,
                                moe_stream_t stream) {
  moe_status st = check_rows(out, kMaxRoutes, kMaxHidden);
  if (st != MOE_OK || (st = check_mx(x)) != MOE_OK) return st;
  if (x->rows != out->rows || x->cols != out->cols) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if ((st = check_ptr(out->data, out->dtype)) != MOE_OK) return st;
  if (!aligned(n_rows, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  MxQuantArgs a = quant_args(x, nullptr, n_rows);
  a.out = const_cast<void*>(out->data);
  a.ld_out = out->ld;
  return cuda_status(launch_mx_restore(a, out->dtype, raw(stream)));
}

moe_status moe_nvfp4_mx_dispatch(const moe_mx* x, int32_t K, const int32_t* inv,
                                 const moe_mx* out, moe_stream_t stream) {
  moe_status st = check_mx(x);
  if (st != MOE_OK || (st = check_routes(x->rows, K)) != MOE_OK) return st;
  if ((st = check_mx(out)) != MOE_OK) return st;
  if (out->rows != (int64_t)x->rows * K || out->cols != x->cols) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0) return MOE_OK;
  if (!inv) return MOE_ERR_INVALID_ARG;
  if (!aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  RowArgs a = {};
  a.T = x->rows;
  a.K = K;
  a.H = padded(x->cols);
  a.inv = inv;
  a.x = x->codes;
  a.out = out->codes;
  return cuda_status(launch_dispatch_mx(a, x->scales, out->scales, raw(stream)));
}

moe_status moe_nvfp4_mx_product(const moe_mx* x, const moe_mx* w, int32_t E,
                                const int32_t* offsets, int32_t dtype, void* out, int64_t ld_out,
                                moe_stream_t stream) {
  return product_impl(x, w, E, offsets, dtype, out, ld_out, -1, stream);
}

moe_status moe_nvfp4_selftest_product_timeout(const moe_mx* x, const moe_mx* w, int32_t E,
                                              const int32_t* offsets, int32_t item, int32_t dtype,
                                              void* out, int64_t ld_out, moe_stream_t stream) {
  if (item < 0) return MOE_ERR_INVALID_ARG;
  return product_impl(x, w, E, offsets, dtype, out, ld_out, item, stream);
}

}  // extern "C"
