// token_loss.cu -- objectives over rows of vocabulary logits z [N][V], each with
// its gradient: the log-probability of a chosen token, the clipped policy loss
// with a KL term, and the KL divergence to a teacher's top logits.
//
// With p = softmax(z / tau) and lse = log sum exp(z / tau):
//   logp     lp = z_a / tau - lse                                  (a: chosen token)
//   policy   r = exp(lp - old);  l = -min(r A, clip(r) A) + b (exp(x) - x - 1),
//            x = ref - lp;  g = dl/dlp = [-r A unless the clipped branch is the
//            smaller] + b (1 - exp(x));  dz_j = w g / tau ([j = a] - p_j)
//   distill  q_i = exp(t_i / tau - L_t), Q = sum_i q_i (L_t: over the teacher's
//            slots, or given);  l = tau^2 sum_i q_i (log q_i - log p_{id_i});
//            dz_j = w tau (Q p_j - sum_{i: id_i = j} q_i)
// So every gradient is a row constant times p_j, plus a few entries.
//
// One block per row, two readings of the row: the running maximum and sum, then
// the gradient.
#include "internal.h"
#include "logits.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float teacher_logit(const TokenLossArgs& a, int64_t i) {
  if (a.t_dtype == kF32) return static_cast<const float*>(a.t_logits)[i];
  const uint16_t* p = static_cast<const uint16_t*>(a.t_logits) + i;
  return a.t_dtype == kBf16 ? load_logit<kBf16>(p) : load_logit<kF16>(p);
}

// What a row adds to its softmax gradient: dz_j = soft p_j, plus `top` at the
// chosen token or -slot_scale q_i at teacher slot i.
struct RowGrad {
  float soft, top, slot_scale;
};

// Loss and gradient of the chosen token's log-probability (policy).
__device__ __forceinline__ float policy_row(const TokenLossArgs& a, int row, float lp,
                                            float* slope) {
  const float A = a.adv[row];
  const float ratio = expf(lp - a.old_logp[row]);
  const float rA = ratio * A;
  const float cA = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi) * A;
  // the comparison is false for a NaN ratio, which then reaches the loss
  float loss = -(cA < rA ? cA : rA);
  float g = cA < rA ? 0.0f : -rA;
  if (a.ref_logp) {
    const float x = a.ref_logp[row] - lp;
    const float em1 = expm1f(x);
    loss += a.kl_coef * (em1 - x);
    g -= a.kl_coef * em1;
  }
  *slope = g;
  return loss;
}

template <int DT, int MODE>
__global__ void __launch_bounds__(kThreads) token_loss_kernel(const TokenLossArgs a) {
  using L = typename LogitType<DT>::type;
  __shared__ MaxSum s_ms[kWarps];
  __shared__ int s_id[kMaxTeacher];
  __shared__ float s_q[kMaxTeacher];
  __shared__ float s_z[kMaxTeacher];
  __shared__ float s_top, s_soft, s_scale;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const L* z = static_cast<const L*>(a.logits) + row * a.ld;
  L* dz = static_cast<L*>(a.dlogits) + row * a.ld_grad;

  const float w = a.row_weight ? a.row_weight[row] : 1.0f;
  int act = -1;
  bool live = w != 0.0f;
  if (MODE != kDistill) {
    act = load_id(a.actions, a.ids64, row);
    live = live && act >= 0 && act < a.V;
  }
  if (!live) {  // left out: the row's logits are not looked at
    if (tid == 0) {
      if (MODE != kTokenLogp) a.row_loss[row] = 0.0f;
      if (MODE != kDistill) a.logp[row] = 0.0f;
    }
    if (a.dlogits)
      for (int j = tid; j < a.V; j += kThreads) store_logit<DT>(dz + j, 0.0f);
    return;
  }

  // the logits at the teacher's slots, read before any gradient is written
  if (MODE == kDistill) {
    if (tid < a.k) {
      const int64_t i = (int64_t)row * a.k + tid;
      const int id = load_id(a.t_ids, a.ids64, i);
      const bool ok = id >= 0 && id < a.V;
      s_id[tid] = ok ? id : -1;
      s_q[tid] = ok ? teacher_logit(a, i) : -INFINITY;
      s_z[tid] = ok ? load_logit<DT>(z + id) : 0.0f;
    }
  } else if (tid == 0) {
    s_z[0] = load_logit<DT>(z + act);
  }

  MaxSum v = {-INFINITY, 0.0f};
  for (int j = tid; j < a.V; j += kThreads) v = merge(v, {load_logit<DT>(z + j), 1.0f}, a.c2);
  v = warp_merge(v, a.c2);
  if (lane == 0) s_ms[warp] = v;
  __syncthreads();
  v = s_ms[0];
  for (int i = 1; i < kWarps; ++i) v = merge(v, s_ms[i], a.c2);
  const float m = finite_ref(v.m);

  if (warp == 0) {
    float loss = 0.0f, soft = 0.0f, top = 0.0f, scale = 0.0f, lp = 0.0f;
    const float ln_s = logf(v.s);
    if (MODE == kDistill) {
      float tm = -INFINITY;
      for (int i = lane; i < a.k; i += 32) tm = fmaxf(tm, s_q[i]);
      tm = finite_ref(warp_max(tm));
      float ts = 0.0f;
      for (int i = lane; i < a.k; i += 32) ts += expf((s_q[i] - tm) * a.inv_tau);
      ts = warp_sum(ts);
      // log q_i = (t_i - tm) / tau + shift
      const float shift = a.t_lse ? tm * a.inv_tau - a.t_lse[row] : -logf(ts);
      float Q = 0.0f, kl = 0.0f;
      for (int i = lane; i < a.k; i += 32) {
        const float lq = (s_q[i] - tm) * a.inv_tau + shift;
        const float q = ts == 0.0f ? 0.0f : expf(lq);
        s_q[i] = q;
        Q += q;
        if (q != 0.0f) kl += q * (lq - (s_z[i] - m) * a.inv_tau + ln_s);
      }
      Q = warp_sum(Q);
      kl = warp_sum(kl);
      if (v.s != 0.0f && Q != 0.0f) {
        loss = a.tau * a.tau * kl;
        soft = w * a.tau * Q;
        scale = w * a.tau;
      }
    } else if (v.s != 0.0f) {
      lp = (s_z[0] - m) * a.inv_tau - ln_s;
      float slope = 0.0f;
      if (MODE == kPolicy) loss = policy_row(a, row, lp, &slope);
      top = w * slope * a.inv_tau;
      soft = -top;
    }
    if (lane == 0) {
      if (MODE != kTokenLogp) a.row_loss[row] = loss;
      if (MODE != kDistill) a.logp[row] = lp;
      s_soft = soft;
      s_top = top;
      s_scale = scale;
    }
  }
  if (!a.dlogits) return;
  __syncthreads();

  // a row without a finite logit or without a teacher has soft = 0: zeros
  const float coef = s_soft == 0.0f ? 0.0f : s_soft / v.s;
  for (int j = tid; j < a.V; j += kThreads) {
    const float p = s_soft == 0.0f ? 0.0f : ex2((load_logit<DT>(z + j) - m) * a.c2);
    store_logit<DT>(dz + j, coef * p);
  }
  __syncthreads();  // the few entries overwrite what the loop stored
  if (MODE == kDistill) {
    if (tid < a.k && s_id[tid] >= 0 && s_scale != 0.0f) {
      float q = 0.0f;  // slots that repeat a token add up, each writing the same sum
      for (int i = 0; i < a.k; ++i) q += s_id[i] == s_id[tid] ? s_q[i] : 0.0f;
      store_logit<DT>(dz + s_id[tid], coef * ex2((s_z[tid] - m) * a.c2) - s_scale * q);
    }
  } else if (tid == 0 && s_soft != 0.0f) {
    store_logit<DT>(dz + act, coef * ex2((s_z[0] - m) * a.c2) + s_top);
  }
}

template <int DT>
cudaError_t launch_dtype(const TokenLossArgs& a, int mode, cudaStream_t s) {
  const dim3 grid(a.N), block(kThreads);
  if (mode == kTokenLogp) return launch_pdl(token_loss_kernel<DT, kTokenLogp>, grid, block, 0, s, a);
  if (mode == kPolicy) return launch_pdl(token_loss_kernel<DT, kPolicy>, grid, block, 0, s, a);
  return launch_pdl(token_loss_kernel<DT, kDistill>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_token_loss(const TokenLossArgs& a, int mode, int dtype, cudaStream_t s) {
  if (dtype == kF32) return launch_dtype<kF32>(a, mode, s);
  if (dtype == kBf16) return launch_dtype<kBf16>(a, mode, s);
  return launch_dtype<kF16>(a, mode, s);
}

}  // namespace moe
