// loss_api.cu -- entry points of the training objectives: argument checks and the
// launch.  No allocation and no host synchronisation.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe_nvfp4.h"
#include "internal.h"
#include "loss.h"

using namespace moe;

namespace {

static_assert((int)MOE_DTYPE_F32 == kF32 && (int)MOE_DTYPE_BF16 == kBf16 &&
              (int)MOE_DTYPE_F16 == kF16, "moe_dtype and LossDtype agree");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
uintptr_t dtype_size(int32_t d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // reported here, not by the next call
  return MOE_ERR_CUDA;
}
bool bool_ok(int32_t b) { return b == 0 || b == 1; }

// Shape of a matrix of logits; its pointer is looked at only when it has rows.
moe_status check_logits(const moe_logits* z, int32_t max_cols) {
  if (!z || z->rows < 0 || z->cols < 1 || !dtype_ok(z->dtype)) return MOE_ERR_INVALID_ARG;
  if (z->cols > max_cols || z->rows > (1 << 26)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (z->ld < z->cols) return MOE_ERR_INVALID_ARG;
  if (z->rows == 0) return MOE_OK;
  if (!z->data) return MOE_ERR_INVALID_ARG;
  return aligned(z->data, dtype_size(z->dtype)) ? MOE_OK : MOE_ERR_MISALIGNED;
}

// A positive temperature whose reciprocal and log2(e) multiple are finite.
bool temperature_ok(float t) { return t >= 1e-30f && t <= 1e30f; }

TokenLossArgs token_args(const moe_logits* z, float temperature, const float* row_weight,
                         void* dlogits, int64_t ld_grad) {
  TokenLossArgs a = {};
  a.N = z->rows;
  a.V = z->cols;
  a.ld = z->ld;
  a.logits = z->data;
  a.tau = temperature;
  a.inv_tau = 1.0f / temperature;
  a.c2 = (float)(1.4426950408889634 / (double)temperature);
  a.row_weight = row_weight;
  a.dlogits = dlogits;
  a.ld_grad = ld_grad;
  return a;
}

// dlogits of a *_grad call.
moe_status check_grad(const moe_logits* z, const void* dlogits, int64_t ld_grad,
                      const float* row_weight) {
  if (ld_grad < z->cols) return MOE_ERR_INVALID_ARG;
  if (z->rows == 0) return MOE_OK;
  if (!dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned(dlogits, dtype_size(z->dtype)) || !aligned(row_weight, 4))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status run(const TokenLossArgs& a, int mode, int dtype, moe_stream_t stream) {
  const int st = device_status(nullptr);
  if (st != MOE_OK) return (moe_status)st;
  return cuda_status(launch_token_loss(a, mode, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status policy_impl(const moe_logits* z, const void* actions, int32_t ids_int64,
                       const float* old_logp, const float* adv, const float* ref_logp,
                       const moe_policy_opts* o, const float* row_weight, float* row_loss,
                       float* logp, void* dlogits, int64_t ld_grad, bool grad,
                       moe_stream_t stream, const LeaveArgs* leave = nullptr) {
  moe_status st = check_logits(z, kMaxVocab);
  if (st != MOE_OK) return st;
  if (!o || !bool_ok(ids_int64) || !(o->clip_low >= 0.0f && o->clip_low <= 1.0f) ||
      !(o->clip_high >= 0.0f && std::isfinite(o->clip_high)) || !std::isfinite(o->kl_coef) ||
      !temperature_ok(o->temperature))
    return MOE_ERR_INVALID_ARG;
  if (grad && (st = check_grad(z, dlogits, ld_grad, row_weight)) != MOE_OK) return st;
  if (z->rows == 0) return MOE_OK;
  if (!actions || !old_logp || !adv || !row_loss || !logp || (o->kl_coef != 0.0f && !ref_logp))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(actions, ids_int64 ? 8 : 4) || !aligned(old_logp, 4) || !aligned(adv, 4) ||
      !aligned(ref_logp, 4) || !aligned(row_loss, 4) || !aligned(logp, 4))
    return MOE_ERR_MISALIGNED;
  TokenLossArgs a = token_args(z, o->temperature, row_weight, dlogits, ld_grad);
  a.actions = actions;
  a.ids64 = ids_int64;
  a.old_logp = old_logp;
  a.adv = adv;
  a.ref_logp = o->kl_coef != 0.0f ? ref_logp : nullptr;  // a term switched off is not 0 * inf
  a.clip_lo = 1.0f - o->clip_low;
  a.clip_hi = 1.0f + o->clip_high;
  a.kl_coef = o->kl_coef;
  a.row_loss = row_loss;
  a.logp = logp;
  if (leave) {
    const int C = token_loss_cluster(z->cols, kBf16);
    if (z->dtype != MOE_DTYPE_BF16 || C == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (leave->rank >= C) return MOE_ERR_INVALID_ARG;
    if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
    return cuda_status(launch_token_loss_leave(a, *leave, reinterpret_cast<cudaStream_t>(stream)));
  }
  return run(a, kPolicy, z->dtype, stream);
}

moe_status distill_impl(const moe_logits* z, const moe_teacher* t, const float* row_weight,
                        float temperature, float* row_loss, void* dlogits, int64_t ld_grad,
                        bool grad, moe_stream_t stream) {
  moe_status st = check_logits(z, kMaxVocab);
  if (st != MOE_OK) return st;
  if (!t || t->K < 1 || !bool_ok(t->ids_int64) || !dtype_ok(t->dtype) ||
      !temperature_ok(temperature))
    return MOE_ERR_INVALID_ARG;
  if (t->K > kMaxTeacher) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (grad && (st = check_grad(z, dlogits, ld_grad, row_weight)) != MOE_OK) return st;
  if (z->rows == 0) return MOE_OK;
  if (!t->ids || !t->logits || !row_loss) return MOE_ERR_INVALID_ARG;
  if (!aligned(t->ids, t->ids_int64 ? 8 : 4) || !aligned(t->logits, dtype_size(t->dtype)) ||
      !aligned(t->lse, 4) || !aligned(row_loss, 4))
    return MOE_ERR_MISALIGNED;
  TokenLossArgs a = token_args(z, temperature, row_weight, dlogits, ld_grad);
  a.ids64 = t->ids_int64;
  a.k = t->K;
  a.t_ids = t->ids;
  a.t_logits = t->logits;
  a.t_dtype = t->dtype;
  a.t_lse = t->lse;
  a.row_loss = row_loss;
  return run(a, kDistill, z->dtype, stream);
}

// Shape limits of the router batch; pointers only when it has rows.
moe_status check_batch(const moe_router_batch* b) {
  if (!b) return MOE_ERR_INVALID_ARG;
  moe_status st = check_logits(&b->logits, 1024);
  if (st != MOE_OK) return st;
  if (b->K < 1 || b->S < 1 || !bool_ok(b->ids_int64) || !std::isfinite(b->balance_coef) ||
      !std::isfinite(b->z_coef) || (!b->seq_offsets && b->S != 1))
    return MOE_ERR_INVALID_ARG;
  if (b->K > 32 || b->K > b->logits.cols || (int64_t)b->logits.rows * b->K > (int64_t(1) << 26) ||
      b->S > (1 << 20) || (int64_t)b->S * b->logits.cols > (int64_t(1) << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (b->logits.rows == 0) return MOE_OK;
  if (!b->topk_ids) return MOE_ERR_INVALID_ARG;
  if (!aligned(b->topk_ids, b->ids_int64 ? 8 : 4) || !aligned(b->seq_offsets, 4))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

RouterLossArgs router_args(const moe_router_batch* b) {
  RouterLossArgs a = {};
  a.T = b->logits.rows;
  a.E = b->logits.cols;
  a.K = b->K;
  a.S = b->S;
  a.ld = b->logits.ld;
  a.logits = b->logits.data;
  a.ids = b->topk_ids;
  a.ids64 = b->ids_int64;
  a.mask = b->token_mask;
  a.offsets = b->seq_offsets;
  a.balance_coef = b->balance_coef;
  a.z_coef = b->z_coef;
  return a;
}

}  // namespace

extern "C" {

moe_status moe_nvfp4_token_logp(const moe_logits* z, const void* actions, int32_t ids_int64,
                                float temperature, float* logp, moe_stream_t stream) {
  moe_status st = check_logits(z, kMaxVocab);
  if (st != MOE_OK) return st;
  if (!bool_ok(ids_int64) || !temperature_ok(temperature)) return MOE_ERR_INVALID_ARG;
  if (z->rows == 0) return MOE_OK;
  if (!actions || !logp) return MOE_ERR_INVALID_ARG;
  if (!aligned(actions, ids_int64 ? 8 : 4) || !aligned(logp, 4)) return MOE_ERR_MISALIGNED;
  TokenLossArgs a = token_args(z, temperature, nullptr, nullptr, 0);
  a.actions = actions;
  a.ids64 = ids_int64;
  a.logp = logp;
  return run(a, kPolicy, z->dtype, stream);
}

moe_status moe_nvfp4_policy_loss(const moe_logits* z, const void* actions, int32_t ids_int64,
                                 const float* old_logp, const float* adv, const float* ref_logp,
                                 const moe_policy_opts* opts, float* row_loss, float* logp,
                                 moe_stream_t stream) {
  return policy_impl(z, actions, ids_int64, old_logp, adv, ref_logp, opts, nullptr, row_loss, logp,
                     nullptr, 0, false, stream);
}

moe_status moe_nvfp4_policy_loss_grad(const moe_logits* z, const void* actions,
                                      int32_t ids_int64, const float* old_logp, const float* adv,
                                      const float* ref_logp, const float* row_weight,
                                      const moe_policy_opts* opts, float* row_loss, float* logp,
                                      void* dlogits, int64_t ld_grad, moe_stream_t stream) {
  return policy_impl(z, actions, ids_int64, old_logp, adv, ref_logp, opts, row_weight, row_loss,
                     logp, dlogits, ld_grad, true, stream);
}

moe_status moe_nvfp4_distill_loss(const moe_logits* z, const moe_teacher* teacher,
                                  float temperature, float* row_loss, moe_stream_t stream) {
  return distill_impl(z, teacher, nullptr, temperature, row_loss, nullptr, 0, false, stream);
}

moe_status moe_nvfp4_distill_loss_grad(const moe_logits* z, const moe_teacher* teacher,
                                       const float* row_weight, float temperature,
                                       float* row_loss, void* dlogits, int64_t ld_grad,
                                       moe_stream_t stream) {
  return distill_impl(z, teacher, row_weight, temperature, row_loss, dlogits, ld_grad, true,
                      stream);
}

moe_status moe_nvfp4_selftest_loss_timeout(const moe_logits* z, const void* actions,
                                           int32_t ids_int64, const float* old_logp,
                                           const float* adv, int32_t role, int32_t rank,
                                           int32_t row, float* row_loss, float* logp,
                                           void* dlogits, int64_t ld_grad, moe_stream_t stream) {
  const moe_policy_opts o = {0.2f, 0.2f, 0.0f, 1.0f};
  const LeaveArgs leave = {role, rank, row};
  if (role < kConsumers || role > kFinish || rank < 0 || row < 0) return MOE_ERR_INVALID_ARG;
  return policy_impl(z, actions, ids_int64, old_logp, adv, nullptr, &o, nullptr, row_loss, logp,
                     dlogits, ld_grad, true, stream, &leave);
}

size_t moe_nvfp4_router_loss_workspace_bytes(int32_t T, int32_t E, int32_t S) {
  if (T < 0 || T > (1 << 26) || E < 1 || E > 1024 || S < 1 || S > (1 << 20) ||
      (int64_t)S * E > (int64_t(1) << 30))
    return 0;
  return router_loss_ws_bytes(T, E, S);
}

moe_status moe_nvfp4_router_loss(const moe_router_batch* b, float* losses, int32_t* counts,
                                 int32_t* tokens, void* ws, size_t ws_bytes,
                                 moe_stream_t stream) {
  moe_status st = check_batch(b);
  if (st != MOE_OK) return st;
  if (!losses || !counts || !tokens || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(losses, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(ws, 256))
    return MOE_ERR_MISALIGNED;
  RouterLossArgs a = router_args(b);
  if (ws_bytes < router_loss_ws_bytes(a.T, a.E, a.S)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.T == 0) {
    cudaError_t e = cudaMemsetAsync(losses, 0, 2 * sizeof(float), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(counts, 0, (size_t)a.S * a.E * sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(tokens, 0, ((size_t)a.S + 1) * sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, kStatusWords * sizeof(int32_t), s);
    return cuda_status(e);
  }
  a.losses = losses;
  a.counts = counts;
  a.tokens = tokens;
  a.ws = ws;
  return cuda_status(launch_router_loss(a, b->logits.dtype, s));
}

moe_status moe_nvfp4_router_loss_grad(const moe_router_batch* b, const int32_t* counts,
                                      const int32_t* tokens, const float* loss_grad,
                                      const float* topk_w, const float* d_topk_w, void* dlogits,
                                      int64_t ld_grad, moe_stream_t stream) {
  moe_status st = check_batch(b);
  if (st != MOE_OK) return st;
  if ((st = check_grad(&b->logits, dlogits, ld_grad, loss_grad)) != MOE_OK) return st;
  if (!topk_w != !d_topk_w) return MOE_ERR_INVALID_ARG;
  if (b->logits.rows == 0) return MOE_OK;
  if (!counts || !tokens) return MOE_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(tokens, 4) || !aligned(topk_w, 4) || !aligned(d_topk_w, 4))
    return MOE_ERR_MISALIGNED;
  if ((st = (moe_status)device_status(nullptr)) != MOE_OK) return st;
  RouterLossArgs a = router_args(b);
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.loss_grad = loss_grad;
  a.topk_w = topk_w;
  a.d_topk_w = d_topk_w;
  a.dlogits = dlogits;
  a.ld_grad = ld_grad;
  return cuda_status(
      launch_router_loss_grad(a, b->logits.dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
