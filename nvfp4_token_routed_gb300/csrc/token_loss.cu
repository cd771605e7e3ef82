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
// What a call cannot do without is one reading of z and, with a gradient, one writing of
// dz; so the row stays on chip between its sum and its gradient, in registers (rows of 16
// KB and less) or in the shared memory of a cluster's blocks (longer ones, loaded ahead by
// bulk copies).  Measured on GB300 against a copy's 6786 GB/s: bf16 gradients of 8192 x
// 131072 logits in 670 us (0.95, distillation) and 632 us (1.0, policy), losses alone of
// 12000 x 32000 f16 logits in 114 us (0.99).  The bound beside memory is instruction issue:
// at two exponentials a bf16 logit and 4 bytes, a reading and a writing leave about 22
// lane instructions a logit, and the kernel takes 12.
#include <climits>
#include <type_traits>

#include "cluster.cuh"
#include "internal.h"
#include "logits.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float teacher_logit(const TokenLossArgs& a, int64_t i) {
  if (a.t_dtype == kF32) return static_cast<const float*>(a.t_logits)[i];
  const uint16_t* p = static_cast<const uint16_t*>(a.t_logits) + i;
  return a.t_dtype == kBf16 ? load_logit<kBf16>(p) : load_logit<kF16>(p);
}

// A row counts unless its weight is 0 or its action is no token.
template <int MODE>
__device__ __forceinline__ bool row_live(const TokenLossArgs& a, int row) {
  bool live = !a.row_weight || a.row_weight[row] != 0.0f;
  if (MODE == kPolicy) {
    const int act = load_id(a.actions, a.ids64, row);
    live = live && act >= 0 && act < a.V;
  }
  return live;
}

// Loss and its slope in the chosen token's log-probability (policy).
__device__ __forceinline__ float policy_row(const TokenLossArgs& a, float lp, float old, float A,
                                            float ref, float* slope) {
  const float ratio = expf(lp - old);
  // a ratio beyond fp32 times no advantage is nothing; a NaN ratio stays one
  const float rA = A == 0.0f && ratio > a.clip_hi ? 0.0f : ratio * A;
  const float cA = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi) * A;
  // the comparison is false for a NaN ratio, which then reaches the loss
  float loss = -(cA < rA ? cA : rA);
  float g = cA < rA ? 0.0f : -rA;
  if (a.ref_logp) {
    const float x = ref - lp;
    const float em1 = expm1f(x);
    loss += a.kl_coef * (em1 - x);
    g -= a.kl_coef * em1;
  }
  *slope = g;
  return loss;
}

// How a row is divided: `head` logits up to the first 16-byte boundary and `tail`
// after the last (the edges, at most 14), between them nb vectors of 16 bytes, `per`
// of them to each of C blocks.
struct Split {
  int head, tail, nb, per;
};
constexpr int kMaxEdge = 14;
template <int DT>
__device__ __forceinline__ Split split_row(const void* row, int V, int C) {
  constexpr int kSize = DT == kF32 ? 4 : 2;
  Split s;
  s.head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kSize);
  s.nb = (V - s.head) / Vec<DT>::kElems;
  s.tail = V - s.head - s.nb * Vec<DT>::kElems;
  s.per = (s.nb + C - 1) / C;
  return s;
}
// Column of edge i.
__device__ __forceinline__ int edge_column(const Split& s, int V, int i) {
  return i < s.head ? i : V - s.tail + (i - s.head);
}

// A row's gradient: vector i of 16 bytes at the logits' boundaries, which are the
// gradient's own where the two rows are aligned alike.
// Where they are not, a vector is stored by the element (6000 x 50257 bf16 gradients of
// rows of 50304: 198 us with a gradient strided alike, 794 with a contiguous one).
template <int DT>
struct GradRow {
  using L = typename LogitType<DT>::type;
  L* body;  // the logit of vector 0
  bool aligned;
  __device__ __forceinline__ uint4* vecs() const { return reinterpret_cast<uint4*>(body); }
  __device__ __forceinline__ void store(int i, const Vec<DT>& g) const {
    if (aligned) {
      vecs()[i] = g.v;
      return;
    }
    L* p = body + (int64_t)i * Vec<DT>::kElems;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = g.word(w);
      if constexpr (DT == kF32) {
        p[w] = __uint_as_float(x);
      } else {
        p[2 * w] = (uint16_t)x;
        p[2 * w + 1] = (uint16_t)(x >> 16);
      }
    }
  }
};
template <int DT>
__device__ __forceinline__ GradRow<DT> grad_row(const void* z, typename LogitType<DT>::type* dz,
                                                int head) {
  return {dz + head,
          ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0};
}

// The dense part of a row's gradient, coef 2^(z c - k) for every logit.  For 16-bit
// gradients the size of coef is folded into the exponent, so that a pair of logits costs
// one multiply-add, two exponentials and one conversion (which takes the sign).  For |k| <
// kFoldRange the sum log2 |coef| - k is below 512 in size (a coef of 2^-149 at the least), so
// its rounding is at most 2^-16, and log2f's own error on |log2 coef| about as much: 2e-5 of
// an entry, below its rounding to 16 bits.  Beyond it a vector at a time, its exponentials
// multiplied by coef: 6000 x 100000 bf16 at temperature 0.1 takes 456 us with |k| = 260 and
// 453 us at temperature 0.11 with |k| = 236.
constexpr float kFoldRange = 256.0f;
struct Soft {
  float coef;  // 0: the gradient is 0
  float m, k;  // reference
  float fold;  // log2 |coef| - k
};
template <int DT>
__device__ __forceinline__ Vec<DT> soft_vec(const Vec<DT>& d, const Soft& r, float c) {
  Vec<DT> g;
  const float b = DT == kF32 ? -r.k : r.fold;
  const f32x2 c2 = pack2(c, c), bias = pack2(b, b);
  const uint32_t sign = r.coef < 0.0f ? 0x80008000u : 0u;
#pragma unroll
  for (int j = 0; j < Vec<DT>::kPairs; ++j) {
    const float2 x = unpack2(fma2(pack2(d.pair(j)), c2, bias));
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    if constexpr (DT == kF32) {
      g.set_pair(j, unpack2(mul2(pack2(r.coef, r.coef), pack2(e))));
    } else {
      g.set_pair(j, e);
      g.set_word(j, g.word(j) ^ sign);
    }
  }
  return g;
}
template <int DT>
__device__ __noinline__ uint4 far_vec(uint4 v, float coef, float m, float c) {
  const Vec<DT> d = {v};
  Vec<DT> g;
#pragma unroll
  for (int j = 0; j < Vec<DT>::kPairs; ++j) {
    const float2 x = d.pair(j);
    g.set_pair(j, make_float2(coef * ex2(exponent(x.x, m, c)), coef * ex2(exponent(x.y, m, c))));
  }
  return g.v;
}
// fn(vector function, std::true_type) for a row whose gradient is dense and near, of
// either sign; fn(vector function, std::false_type) for one that is 0 (clipped, no
// teacher, or no finite logit) or far.
template <int DT, typename F>
__device__ __forceinline__ void with_soft(const Soft& r, float c, F fn) {
  const bool near = DT == kF32 ? near_ref(r.k) : fabsf(r.k) < kFoldRange;
  if (r.coef == 0.0f || !near) {
    fn([&](const Vec<DT>& d) {
      Vec<DT> g;
      if (r.coef == 0.0f) g.fill(0);
      else g.v = far_vec<DT>(d.v, r.coef, r.m, c);
      return g;
    }, std::false_type{});
  } else {
    fn([&](const Vec<DT>& d) { return soft_vec<DT>(d, r, c); }, std::true_type{});
  }
}
__device__ __forceinline__ float soft_at(float z, const Soft& r, float c) {
  return r.coef == 0.0f ? 0.0f : r.coef * ex2(exponent(z, r.m, c));
}

// What a teacher's slots say without the student's normaliser, by one warp: q into
// s_q (which holds the teacher's logits), Q = sum q, and kl, zr with
//   sum q_i (log q_i - log p_i) = kl + Q (log s - log weight of zr),
// zr the largest of the student's logits at the slots; -inf: none is finite, and kl is
// without it.
struct TeacherSums {
  float Q, kl, zr;
};
__device__ __forceinline__ TeacherSums teacher_sums(const TokenLossArgs& a, int row, int lane,
                                                    float* s_q, const float* s_z) {
  float tm = -INFINITY, zr = -INFINITY;
  for (int i = lane; i < a.k; i += 32) {
    tm = fmaxf(tm, s_q[i]);
    zr = fmaxf(zr, s_z[i]);
  }
  tm = finite_ref(warp_max(tm));
  zr = warp_max(zr);
  const float base = finite_ref(zr);
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
    if (q != 0.0f) kl += q * (lq - (s_z[i] - base) * a.inv_tau);
  }
  return {warp_sum(Q), warp_sum(kl), zr};
}

// A row's teacher slots, spread over NT threads: ids (-1: empty), the teacher's logits
// and the student's at those tokens.  All ids are loaded before the first logit.
template <int DT, int NT>
struct TeacherSlots {
  static constexpr int U = (kMaxTeacher + NT - 1) / NT;
  int id[U];
  float t[U], z[U];
  __device__ __forceinline__ void load_ids(const TokenLossArgs& a, int row, int tid) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      id[u] = -1;
      t[u] = 0.0f;
      if (NT * u >= a.k) continue;
      const int i = tid + NT * u;
      const int64_t at = (int64_t)row * a.k + i;
      if (i < a.k) {
        id[u] = load_id(a.t_ids, a.ids64, at);
        t[u] = teacher_logit(a, at);
      }
    }
  }
  __device__ __forceinline__ void load_logits(const TokenLossArgs& a,
                                              const typename LogitType<DT>::type* z_row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      z[u] = -INFINITY;
      if (NT * u >= a.k) continue;
      if (id[u] >= a.V) id[u] = -1;
      if (id[u] >= 0) z[u] = load_logit<DT>(z_row + id[u]);
    }
  }
  // s_id may be null.
  __device__ __forceinline__ void write(int k, int tid, int* s_id, float* s_t, float* s_z) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = tid + NT * u;
      if (i >= k) break;
      if (s_id) s_id[i] = max(id[u], -1);
      s_t[i] = id[u] >= 0 ? t[u] : -INFINITY;
      s_z[i] = z[u];
    }
  }
};

// The slots whose token may be an earlier slot's too, by one warp: bit i % 32 of
// s_again[i / 32].  A hash of the tokens seen decides; it may name a slot too many.
constexpr int kSeenWords = 256;  // 8192 bits: a false name every fourth row at 64 slots
__device__ __forceinline__ void name_repeats(int k, int lane, const int* s_id, uint32_t* s_seen,
                                             uint32_t* s_again) {
  for (int i = lane; i < kSeenWords; i += 32) s_seen[i] = 0;
  __syncwarp();
  for (int i = lane; i - lane < k; i += 32) {
    const int id = i < k ? s_id[i] : -1;
    const uint32_t h = ((uint32_t)id * 2654435761u) >> 19, bit = 1u << (h & 31);
    const bool again = id >= 0 && (atomicOr(&s_seen[h >> 5], bit) & bit);
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, again);
    if (lane == 0) s_again[i / 32] = all;
  }
  __syncwarp();
}
// fn(slot, sum of q over the slots of its token) for each of them, by one warp.
template <typename F>
__device__ __forceinline__ void for_repeats(int k, int lane, const int* s_id, const float* s_q,
                                            const uint32_t* s_again, F fn) {
  for (int u = 0; 32 * u < k; ++u) {
    for (uint32_t m = s_again[u]; m; m &= m - 1) {
      const int slot = 32 * u + __ffs(m) - 1, id = s_id[slot];
      float part = 0.0f;
      for (int i = lane; i < k; i += 32) part += s_id[i] == id ? s_q[i] : 0.0f;
      fn(slot, warp_sum(part));
    }
  }
}

// A row's results once its largest logit and sum v are known.
struct RowResult {
  Soft soft;    // dz_j = soft_j ...
  float top;    // ... + top at the chosen token (policy)
  float scale;  // ... - scale q_i at teacher slot i (distill)
  float loss, logp;
};
template <int MODE>
__device__ __forceinline__ RowResult finish_row(const TokenLossArgs& a, MaxSum v, float w,
                                                const TeacherSums& t, float z_act, float old,
                                                float adv, float ref) {
  const float m = finite_ref(v.m);
  RowResult r = {{0.0f, m, ref_exponent(m, a.c2), 0.0f}, 0.0f, 0.0f, 0.0f, 0.0f};
  if (v.s == 0.0f) return r;  // no finite logit
  const float ln_s = logf(v.s);
  float soft = 0.0f;
  if (MODE == kDistill) {
    if (t.Q == 0.0f) return r;  // no teacher
    const float lw = t.zr == -INFINITY ? 0.0f : log_weight(t.zr, m, a.c2, a.inv_tau);
    r.loss = a.tau * a.tau * (t.kl + t.Q * (ln_s - lw));
    soft = w * a.tau * t.Q;
    r.scale = w * a.tau;
  } else {
    // a token that is the whole sum: 0
    r.logp = ex2(exponent(z_act, m, a.c2)) >= v.s
                 ? 0.0f
                 : log_weight(z_act, m, a.c2, a.inv_tau) - ln_s;
    float slope = 0.0f;
    if (a.adv) r.loss = policy_row(a, r.logp, old, adv, ref, &slope);
    r.top = w * slope * a.inv_tau;
    soft = -r.top;
  }
  if (soft != 0.0f) {
    r.soft.coef = soft / v.s;
    r.soft.fold = log2f(fabsf(r.soft.coef)) - r.soft.k;
  }
  return r;
}

// ---------------------------------------------------------------- short rows
//
// NT threads a row, each with VPT vectors of it in registers: one warp (rows of 2 KB and
// less, no block-wide wait), or a block of 64 to 256.  Many small blocks an SM overlap
// one's loads with another's reductions; a row's latency is what bounds them (16384 bf16
// rows of 4096, policy gradient: 60 us, 0.66 of the copy rate; of 1000: 21 us, 0.47; fp32
// rows of 4096: 78 us, 1.0).  Persistent blocks with the next row in registers took 117 of
// them and 76 us for the first of these.

constexpr int short_rows_per_block(int NT) { return NT == 32 ? 8 : 1; }
// Threads an SM is to hold, 64 registers each: without the bound the compiler takes up to
// 110 (distillation of 16384 x 4096: 116 us, with it 74, with room for 1280 threads 84).
constexpr int kShortResident = 1024;

template <int DT, int MODE, int NT, int VPT>
__global__ void __launch_bounds__(NT * short_rows_per_block(NT),
                                  kShortResident / (NT * short_rows_per_block(NT)))
    short_row_kernel(const TokenLossArgs a) {
  using L = typename LogitType<DT>::type;
  using V16 = Vec<DT>;
  constexpr int kWarps = NT / 32, kRows = short_rows_per_block(NT);
  constexpr int kSlots = MODE == kDistill ? kMaxTeacher : 1;
  struct Shared {
    MaxSum ms[kWarps];
    int id[kSlots];
    float q[kSlots], z[kSlots];
    uint32_t seen[MODE == kDistill ? kSeenWords : 1], again[kMaxTeacher / 32];
    TeacherSums t;
    RowResult r;
  };
  __shared__ Shared shared[kRows];
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x / NT, tid = threadIdx.x % NT, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x * kRows + sub;
  if (row >= a.N) return;
  Shared& sh = shared[sub];
  auto sync = [] {  // the row's threads
    if (NT == 32) __syncwarp();
    else __syncthreads();
  };
  const L* z = static_cast<const L*>(a.logits) + row * a.ld;
  L* dz = static_cast<L*>(a.dlogits) + row * a.ld_grad;
  const Split sp = split_row<DT>(z, a.V, 1);
  const int edge = tid < sp.head + sp.tail ? edge_column(sp, a.V, tid) : -1;
  const uint4* zv = reinterpret_cast<const uint4*>(z + sp.head);
  const GradRow<DT> out = grad_row<DT>(z, dz, sp.head);
  auto store_zeros = [&] {
    V16 zero;
    zero.fill(0);
    for (int i = tid; i < sp.nb; i += NT) out.store(i, zero);
    if (edge >= 0) store_logit<DT>(dz + edge, 0.0f);
  };
  if (!row_live<MODE>(a, row)) {  // left out: the row's logits are not looked at
    if (tid == 0) {
      if (a.row_loss) a.row_loss[row] = 0.0f;
      if (a.logp) a.logp[row] = 0.0f;
    }
    if (a.dlogits) store_zeros();
    return;
  }

  V16 d[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = i * NT + tid;
    if (at < sp.nb) d[i].v = zv[at];
    else d[i].fill(V16::kNegInf);
  }
  const float x_edge = edge >= 0 ? load_logit<DT>(z + edge) : -INFINITY;

  // the few logits that the loss picks out, read before any gradient is written
  int act = -1;
  float w = 1.0f, old = 0.0f, adv = 0.0f, ref = 0.0f, z_act = 0.0f;
  if constexpr (MODE == kDistill) {
    TeacherSlots<DT, NT> few;
    few.load_ids(a, row, tid);
    few.load_logits(a, z);
    few.write(a.k, tid, sh.id, sh.q, sh.z);
  }
  if (tid == 0) {
    if (a.row_weight) w = a.row_weight[row];
    if (MODE == kPolicy) {
      act = load_id(a.actions, a.ids64, row);
      z_act = load_logit<DT>(z + act);
      if (a.adv) {
        old = a.old_logp[row];
        adv = a.adv[row];
        ref = a.ref_logp ? a.ref_logp[row] : 0.0f;
      }
    }
  }
  MaxSum v = add_vecs<DT, VPT>(one_logit(x_edge, a.c2), d, a.c2);
  v = warp_merge(v, a.c2, 32);
  if (kWarps > 1 && lane == 0) sh.ms[warp] = v;
  sync();
  if (MODE == kDistill) {
    if (warp == kWarps - 1) {
      const TeacherSums t = teacher_sums(a, row, lane, sh.q, sh.z);
      if (lane == 0) sh.t = t;
      __syncwarp();
      if (a.dlogits) name_repeats(a.k, lane, sh.id, sh.seen, sh.again);
    }
    sync();
  }
  if (warp == 0) {
    if (kWarps > 1) {
      v = lane < kWarps ? sh.ms[lane] : MaxSum{-INFINITY, 0.0f};
      v = warp_merge(v, a.c2, kWarps);
    }
    if (lane == 0) {
      const RowResult r = finish_row<MODE>(a, v, w, MODE == kDistill ? sh.t : TeacherSums{}, z_act,
                                           old, adv, ref);
      if (a.row_loss) a.row_loss[row] = r.loss;
      if (a.logp) a.logp[row] = r.logp;
      sh.r = r;
    }
  }
  if (!a.dlogits) return;
  sync();

  const RowResult r = sh.r;
  with_soft<DT>(r.soft, a.c2, [&](auto grad_vec, auto) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) d[i] = grad_vec(d[i]);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int at = i * NT + tid;
      if (at < sp.nb) out.store(at, d[i]);
    }
  });
  if (edge >= 0) store_logit<DT>(dz + edge, soft_at(x_edge, r.soft, a.c2));
  if (r.soft.coef == 0.0f) return;
  sync();  // the few entries overwrite what the threads stored
  if (MODE == kDistill) {
    for (int i = tid; i < a.k; i += NT) {
      const int id = sh.id[i];
      if (id >= 0)
        store_logit<DT>(dz + id, soft_at(sh.z[i], r.soft, a.c2) - r.scale * sh.q[i]);
    }
    sync();
    if (warp == 0)
      for_repeats(a.k, lane, sh.id, sh.q, sh.again, [&](int i, float q) {
        if (lane == 0)
          store_logit<DT>(dz + sh.id[i], soft_at(sh.z[i], r.soft, a.c2) - r.scale * q);
      });
  } else if (tid == 0) {
    store_logit<DT>(dz + act, soft_at(z_act, r.soft, a.c2) + r.top);
  }
}

// ---------------------------------------------------------------- long rows
//
// Persistent clusters of C blocks, one block per SM; a block has its C-th part of
// each row.  Roles, which meet at mbarriers only:
//   consumers (2 or 3 groups of 8 warps, rows in turn)  pass 1: running reference and
//                         sum of the block's part, from shared memory; pass 2: its
//                         gradient, from shared memory
//   producer (1 warp)     bulk copies of the part's 16 KB chunks into a ring, as far
//                         ahead as the ring has room
//   gather (3 or 4 warps, rows in turn)  ahead of the consumers the few logits that the
//                         loss picks out, the row's edges and the teacher's side; after
//                         pass 2 the gradient's edges and few entries
//   finish (1 warp a group)  joins the warps' sums, exchanges them within the cluster
//                         (every block gets every other's pair), loss and gradient
//                         constants
// A group's rows always meet the same finish warp, and a slot's rows the same gather
// warp, group and finish warp, so that each waits on a barrier phase by phase.
// One group's waits for the exchange are the other's time to compute: one group of 16
// warps that took pass 1 of the next row before pass 2 spent 785 us on 8192 x 131072, two
// groups of 8 653.  Two groups' parts of 64 KB leave 80 KB of the ring to load ahead; a
// third group left 16 KB and took 877 us, but helps where there is no gradient (12000 x
// 32000: 138 us with two, 109 with three).  Rows that are
// left out pass through no ring slot and no barrier.  All waits are bounded; a role
// whose wait runs out leaves, and soon the others do.  Each tells rank 0 the row it gave up;
// from the first of these on, a row may lack its gradient in any block, whatever its loss:
// at the end the cluster's rows from there on get NaN losses and log-probabilities.

constexpr int kGroupWarps = 8;
constexpr int kGroupThreads = kGroupWarps * 32;
// Groups: with a gradient two, whose parts stay in the ring until pass 2; without, a
// chunk is free again after pass 1, and a third group hides more of the other waits.
// Slots of rows gathered ahead: multiples of the groups and of the gather warps.
constexpr int groups_of(bool grad) { return grad ? 2 : 3; }
constexpr int gather_warps(bool grad) { return grad ? 4 : 3; }
constexpr int slots_of(bool grad) { return grad ? 4 : 6; }
constexpr int long_threads(bool grad) {
  return (groups_of(grad) * (kGroupWarps + 1) + 1 + gather_warps(grad)) * 32;
}
constexpr int kChunkVecs = 1024;  // 16 KB
constexpr int kChunks = 13;
constexpr int kPartsAhead = 16;   // more parts than the ring may hold
constexpr int kMaxCluster = 8;
constexpr int kRingBytes = kChunks * kChunkVecs * 16;

template <int MODE, bool kGrad>
struct Slot {  // a row: what the gather warp prepares, and what comes of it
  static constexpr int kIds = MODE == kDistill && kGrad ? kMaxTeacher : 1;
  static constexpr int kFew = MODE == kDistill ? kMaxTeacher : 1;
  int id[kIds];
  float q[kFew], z[kFew];
  uint32_t seen[MODE == kDistill && kGrad ? kSeenWords : 1], again[kMaxTeacher / 32];
  float edge[kMaxEdge];
  float in[4];  // weight; policy: old log-probability, advantage, reference
  TeacherSums t;
  Soft soft;    // the finish warp's
  float top, scale;
};

template <int MODE, bool kGrad>
struct LongShared {
  static constexpr int kGroups = groups_of(kGrad), kSlots = slots_of(kGrad);
  // A block may send the sums of a group's next row before another has read the last
  // ones, but not those of the row after that, as it has then had the other's next.
  static constexpr int kExchanges = 2 * kGroups;
  Slot<MODE, kGrad> slot[kSlots];
  MaxSum ms[kGroups][kGroupWarps];
  alignas(16) MaxSum cl[kExchanges][kMaxCluster];
  alignas(8) uint64_t full[kPartsAhead], empty[kChunks];
  uint64_t sums[kGroups], go[kGroups], xch[kExchanges];
  uint64_t ready[kSlots];  // gathered
  uint64_t over[kSlots];   // read for the last time: pass 2 done, or without one the loss
  volatile int unloaded;    // the first row that the producer gave up
  volatile int unfinished;  // rank 0's: the first row of the cluster that a role gave up
};

// The rows of one cluster in order, 32 at a time: which of them count.
template <int MODE>
struct RowWalk {
  int first, step, N, lane;
  uint32_t mask;
  __device__ __forceinline__ bool live(const TokenLossArgs& a, int it) {
    if ((it & 31) == 0) {
      const int64_t r = first + (int64_t)(it + lane) * step;
      mask = __ballot_sync(0xFFFFFFFFu, r < N && row_live<MODE>(a, (int)r));
    }
    return (mask >> (it & 31)) & 1;
  }
};

// A place in the ring of chunks: its slot, and the parity of the slot's phase.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kChunks) {
      slot = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void skip(int chunks) {  // at most kChunks
    slot += chunks;
    if (slot >= kChunks) {
      slot -= kChunks;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), parity));
}

// NaN for the cluster's rows from `row` on.
__device__ __noinline__ void mark_unfinished(float* row_loss, float* logp, int row, int N) {
  const int step = gridDim.x / cluster_size();
  for (row += threadIdx.x * step; row < N; row += blockDim.x * step) {
    if (row_loss) row_loss[row] = NAN;
    if (logp) logp[row] = NAN;
  }
}

// kTest: a role of cluster 0 leaves as if a wait had run out.
template <int DT, int MODE, bool kGrad, bool kTest>
__global__ void __launch_bounds__(long_threads(kGrad), 1)
    long_row_kernel(const TokenLossArgs a, const LeaveArgs leave) {
  using L = typename LogitType<DT>::type;
  using V16 = Vec<DT>;
  constexpr int kGroups = groups_of(kGrad), kSlots = slots_of(kGrad);
  constexpr int kGatherWarps = gather_warps(kGrad);
  constexpr int kConsumerWarps = kGroups * kGroupWarps;
  static_assert(kSlots % kGroups == 0 && kSlots % kGatherWarps == 0, "one user a slot");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ LongShared<MODE, kGrad> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster_size(), rank = cluster_rank();
  if (tid == 0) {
    for (int i = 0; i < kPartsAhead; ++i) mbar_init(smem_u32(&sh.full[i]), 1);
    for (int i = 0; i < kChunks; ++i) mbar_init(smem_u32(&sh.empty[i]), kGroupWarps);
    for (int p = 0; p < kGroups; ++p) {
      mbar_init(smem_u32(&sh.sums[p]), kGroupWarps);
      mbar_init(smem_u32(&sh.go[p]), 1);
    }
    for (int p = 0; p < sh.kExchanges; ++p) mbar_init(smem_u32(&sh.xch[p]), 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sh.ready[i]), 1);
      mbar_init(smem_u32(&sh.over[i]), kGrad ? kGroupWarps : 1);
    }
    sh.unloaded = sh.unfinished = INT_MAX;
    fence_barrier_init();
  }
  __syncthreads();
  cluster_arrive();  // before any block writes to another's barrier or memory
  cluster_wait();
  pdl_wait();
  pdl_trigger();

  const int first = blockIdx.x / C, step = gridDim.x / C;
  RowWalk<MODE> walk = {first, step, a.N, lane, 0u};
  const int rows = first < a.N ? (a.N - 1 - first) / step + 1 : 0;
  auto logits_of = [&](int row) { return static_cast<const L*>(a.logits) + row * a.ld; };
  auto grad_of = [&](int row) { return static_cast<L*>(a.dlogits) + row * a.ld_grad; };
  // this block's vectors of a row: [v0, v0 + nv)
  struct Part {
    Split sp;
    int v0, nv, chunks;
  };
  // rows a multiple of 16 bytes apart are divided alike
  const bool alike = a.ld * (DT == kF32 ? 4 : 2) % 16 == 0;
  Part common = {};
  auto part_of = [&](int row) {
    if (alike && row != first) return common;
    Part p;
    p.sp = split_row<DT>(logits_of(row), a.V, C);
    p.v0 = rank * p.sp.per;
    p.nv = max(0, min(p.sp.nb, p.v0 + p.sp.per) - p.v0);
    p.chunks = (p.nv + kChunkVecs - 1) / kChunkVecs;
    return p;
  };
  common = part_of(first);
  int lost = INT_MAX;  // the first row that this warp's role gave up; none: one beyond the last
  auto leaves = [&](int role, int row) {
    return kTest && first == 0 && rank == leave.rank && role == leave.role && row >= leave.row;
  };

  if (warp < kConsumerWarps) {
    constexpr int kPer = kChunkVecs / kGroupThreads;  // vectors of a chunk a thread has
    const int g = warp / kGroupWarps, gtid = tid - g * kGroupThreads;
    RingPos pos;      // of the next row's part
    uint32_t lv = 0;  // live rows passed
    // fn(array of a thread's vectors, their chunk, first vector, vectors left, whether it
    // is the chunk's last call) over a part: a chunk at a time, the last one with as few
    // vectors a thread as it needs; where `whole` is false always with one
    auto steps = [&](int nv, RingPos at, auto whole, auto fn) {
      int left = nv;
      if constexpr (decltype(whole)::value) {
        for (; left > kChunkVecs / 2; left -= kChunkVecs, at.next()) {
          V16 d[kPer];
          fn(d, at.slot, nv - left, left, true);
        }
        if (left > kChunkVecs / 4) {
          V16 d[kPer / 2];
          fn(d, at.slot, nv - left, left, true);
        } else if (left > 0) {
          V16 d[kPer / 4];
          fn(d, at.slot, nv - left, left, true);
        }
      } else {
        for (int q = 0; left > 0; left -= kGroupThreads) {
          V16 d[1];
          const bool last = q == kPer - 1 || left <= kGroupThreads;
          fn(d, at.slot, nv - left, left, last);
          if (++q == kPer) {
            q = 0;
            at.next();
          }
        }
      }
    };
    auto read = [&](auto& d, int slot, int from) {
      const uint4* r =
          reinterpret_cast<const uint4*>(ring) + slot * kChunkVecs + from % kChunkVecs + gtid;
#pragma unroll
      for (int u = 0; u < (int)(sizeof(d) / sizeof(V16)); ++u) d[u].v = r[u * kGroupThreads];
    };
    // Gives a chunk back once the vectors read from it have arrived in registers: the
    // barrier's address takes a word of each (and itself again, so nothing is added).  An
    // arrival alone does not wait for loads in flight, and the next copy into the chunk is
    // not ordered behind them: with the load pipe busy it overtook them.
    auto word_of = [](const auto& d) {
      uint32_t w = 0;
#pragma unroll
      for (int u = 0; u < (int)(sizeof(d) / sizeof(V16)); ++u) w ^= d[u].v.x;
      return w;
    };
    auto release = [&](int slot, uint32_t w) {
      const uint32_t same = __shfl_sync(0xFFFFFFFFu, w, 0);
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[slot]) + (same ^ w));
    };
    int it = 0;
    for (; it < rows; ++it) {
      const int row = first + it * step;
      const bool live = walk.live(a, it);
      const Part p = part_of(row);
      if (!live) {
        if (kGrad && it % kGroups == g) {
          const GradRow<DT> out = grad_row<DT>(logits_of(row), grad_of(row), p.sp.head);
          V16 zero;
          zero.fill(0);
          for (int i = gtid; i < p.nv; i += kGroupThreads) out.store(p.v0 + i, zero);
        }
        continue;
      }
      const uint32_t l = lv++;
      const RingPos at = pos;
      pos.skip(p.chunks);
      if (l % kGroups != g) continue;
      const uint32_t ph = (l / kGroups) & 1;

      MaxSum v = {-INFINITY, 0.0f};
      if (!warp_wait(&sh.full[l % kPartsAhead], (l / kPartsAhead) & 1)) break;
      steps(p.nv, at, std::true_type{}, [&](auto& d, int slot, int from, int left, bool) {
        constexpr int U = sizeof(d) / sizeof(V16);
        read(d, slot, from);
        const uint32_t w = word_of(d);
        if (left < U * kGroupThreads) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (gtid + u * kGroupThreads >= left) d[u].fill(V16::kNegInf);
        }
        v = add_vecs<DT, U>(v, d, a.c2);
        if (!kGrad) release(slot, w);
      });
      v = warp_merge(v, a.c2, 32);
      if (lane == 0) {
        sh.ms[g][warp - g * kGroupWarps] = v;
        mbar_arrive(smem_u32(&sh.sums[g]));
      }

      if (leaves(kConsumers, row) || !warp_wait(&sh.go[g], ph)) break;
      if constexpr (!kGrad) continue;
      const GradRow<DT> out = grad_row<DT>(logits_of(row), grad_of(row), p.sp.head);
      with_soft<DT>(sh.slot[l % kSlots].soft, a.c2, [&](auto grad_vec, auto whole) {
        steps(p.nv, at, whole, [&](auto& d, int slot, int from, int left, bool last) {
          constexpr int U = sizeof(d) / sizeof(V16);
          read(d, slot, from);  // beyond the part: what the slot held, not stored
          const uint32_t w = word_of(d);
          const int base = p.v0 + from + gtid;
#pragma unroll
          for (int u = 0; u < U; ++u) d[u] = grad_vec(d[u]);
          if (last) release(slot, w);
          if (out.aligned && left >= U * kGroupThreads) {
#pragma unroll
            for (int u = 0; u < U; ++u) out.vecs()[base + u * kGroupThreads] = d[u].v;
          } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (gtid + u * kGroupThreads < left) out.store(base + u * kGroupThreads, d[u]);
          }
        });
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.over[l % kSlots]));
    }
    lost = first + it * step;
  } else if (warp == kConsumerWarps) {  // producer
    RingPos pos;
    uint32_t lv = 0;
    bool ok = true;
    int it = 0;
    for (; it < rows; ++it) {
      const int row = first + it * step;
      if (!walk.live(a, it)) continue;
      const Part p = part_of(row);
      const uint4* src = reinterpret_cast<const uint4*>(logits_of(row) + p.sp.head) + p.v0;
      uint64_t* full = &sh.full[lv % kPartsAhead];
      for (int left = p.nv; left > 0; left -= kChunkVecs, pos.next()) {
        ok = !leaves(kProducer, row) && warp_wait(&sh.empty[pos.slot], pos.phase ^ 1);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bytes = 16u * min(kChunkVecs, left);
          // one arrival a part, with its last chunk: the bytes before it are counted too
          if (left <= kChunkVecs) mbar_expect_tx(smem_u32(full), bytes);
          else mbar_add_tx(smem_u32(full), bytes);
          bulk_load(smem_u32(ring) + pos.slot * kChunkVecs * 16, src + (p.nv - left), bytes,
                    smem_u32(full));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (p.nv == 0 && lane == 0) mbar_arrive(smem_u32(full));
      ++lv;
    }
    // no copy may be in flight when the block ends: a part that a wait cut short completes
    // with the chunks it has, and its row is not valid
    lost = first + it * step;
    if (!ok && lane == 0) {
      sh.unloaded = it;
      __threadfence_block();
      mbar_arrive(smem_u32(&sh.full[lv % kPartsAhead]));
    }
    const uint32_t parts = ok ? lv : lv + 1;
    for (uint32_t i = parts > kPartsAhead ? parts - kPartsAhead : 0; i < parts; ++i)
      warp_wait(&sh.full[i % kPartsAhead], (i / kPartsAhead) & 1);
  } else if (warp <= kConsumerWarps + kGatherWarps) {  // gather
    const int g = warp - kConsumerWarps - 1;
    int it = 0;
    uint32_t lv = 0;
    auto next_row = [&] {  // this warp's, or -1
      while (it < rows) {
        const int row = first + it * step;
        if (walk.live(a, it++) && lv++ % kGatherWarps == g) return row;
      }
      return -1;
    };
    // a row's loads, in flight while the row before it is waited for
    TeacherSlots<DT, 32> few;
    int act = 0;
    float x_edge = 0.0f, x_act = 0.0f, in = 0.0f;
    auto fetch = [&](int row, auto meanwhile) {
      const L* z = logits_of(row);
      const Split sp = part_of(row).sp;
      x_edge = lane < sp.head + sp.tail ? load_logit<DT>(z + edge_column(sp, a.V, lane)) : 0.0f;
      if (MODE == kDistill) {
        few.load_ids(a, row, lane);
        in = a.row_weight ? a.row_weight[row] : 1.0f;
        meanwhile();
        few.load_logits(a, z);
      } else {
        const float* from = lane == 0   ? a.row_weight
                            : lane == 1 ? a.old_logp
                            : lane == 2 ? a.adv
                            : lane == 3 ? a.ref_logp
                                        : nullptr;
        in = from ? from[row] : 1.0f;
        if (lane == 0) {
          act = load_id(a.actions, a.ids64, row);
          x_act = load_logit<DT>(z + act);
        }
      }
    };
    int row = next_row();
    if (row >= 0) fetch(row, [] {});
    for (uint32_t l = lv - 1; row >= 0; l = lv - 1) {
      const int i = l % kSlots;
      const uint32_t ph = (l / kSlots) & 1;
      Slot<MODE, kGrad>& s = sh.slot[i];
      if (!kGrad && !warp_wait(&sh.over[i], ph ^ 1)) {
        lost = row;
        break;
      }
      if constexpr (MODE == kDistill) {
        few.write(a.k, lane, kGrad ? s.id : nullptr, s.q, s.z);
        __syncwarp();
        const TeacherSums t = teacher_sums(a, row, lane, s.q, s.z);
        if (lane == 0) {
          s.t = t;
          s.in[0] = in;
        }
      } else {
        if (lane < 4) s.in[lane] = in;
        if (lane == 0) {
          s.id[0] = act;
          s.z[0] = x_act;
        }
      }
      if (lane < kMaxEdge) s.edge[lane] = x_edge;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.ready[i]));
      const int last = row;
      row = next_row();
      auto name = [&] {
        if (MODE == kDistill && kGrad) name_repeats(a.k, lane, s.id, s.seen, s.again);
      };
      if (row >= 0) fetch(row, name);
      else name();
      if constexpr (kGrad) {
        if (leaves(kGather, last) || !warp_wait(&sh.over[i], ph)) {
          lost = last;
          break;
        }
        const Soft soft = s.soft;
        const Part p = part_of(last);  // whose pass 2 is done
        L* dz = grad_of(last);
        if (rank == 0 && lane < p.sp.head + p.sp.tail)
          store_logit<DT>(dz + edge_column(p.sp, a.V, lane), soft_at(s.edge[lane], soft, a.c2));
        __syncwarp();
        if (soft.coef == 0.0f) continue;
        auto store_entry = [&](int j, float more) {
          const int id = s.id[j];
          if (id < 0) return;
          const int e = id - p.sp.head;  // rank 0 has the edges, else whose vector it is
          const int vec = e / V16::kElems - p.v0;
          const bool mine = e < 0 || e >= p.sp.nb * V16::kElems ? rank == 0 : vec >= 0 && vec < p.nv;
          if (mine) store_logit<DT>(dz + id, soft_at(s.z[j], soft, a.c2) + more);
        };
        if (MODE == kDistill) {
          for (int j = lane; j < a.k; j += 32) store_entry(j, -s.scale * s.q[j]);
          __syncwarp();
          for_repeats(a.k, lane, s.id, s.q, s.again, [&](int j, float q) {
            if (lane == 0) store_entry(j, -s.scale * q);
          });
        } else if (lane == 0) {
          store_entry(0, s.top);
        }
        __syncwarp();
      }
    }
  } else {  // finish
    const int b = warp - (kConsumerWarps + 1 + kGatherWarps);  // its group
    uint32_t lv = 0;
    int it = 0;
    for (; it < rows; ++it) {
      const int row = first + it * step;
      if (!walk.live(a, it)) {
        if (rank == 0 && it % kGroups == b) {
          if (lane == 0) {
            if (a.row_loss) a.row_loss[row] = 0.0f;
            if (a.logp) a.logp[row] = 0.0f;
          }
          if (kGrad) {
            const Split sp = part_of(row).sp;
            if (lane < sp.head + sp.tail)
              store_logit<DT>(grad_of(row) + edge_column(sp, a.V, lane), 0.0f);
          }
        }
        continue;
      }
      const uint32_t l = lv++;
      if (l % kGroups != b) continue;
      const int i = l % kSlots, x = l % sh.kExchanges;
      Slot<MODE, kGrad>& s = sh.slot[i];
      const Part p = part_of(row);
      if (leaves(kFinish, row) || !warp_wait(&sh.ready[i], (l / kSlots) & 1) ||
          !warp_wait(&sh.sums[b], (l / kGroups) & 1) || it >= sh.unloaded)
        break;
      // the consumer warps' pairs, and rank 0's edges
      MaxSum v = lane < kGroupWarps ? sh.ms[b][lane] : MaxSum{-INFINITY, 0.0f};
      if (rank == 0 && lane < p.sp.head + p.sp.tail)
        v = merge(v, one_logit(s.edge[lane], a.c2), a.c2);
      v = warp_merge(v, a.c2, 16);
      if (C > 1) {
        if (lane == 0) mbar_expect_tx(smem_u32(&sh.xch[x]), 8u * C);
        __syncwarp();
        if (lane < C)
          st_async_f32x2(smem_u32(&sh.cl[x][rank]), smem_u32(&sh.xch[x]), lane, v.m, v.s);
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait_cluster(smem_u32(&sh.xch[x]), (l / sh.kExchanges) & 1)))
          break;
        v = lane < C ? sh.cl[x][lane] : MaxSum{-INFINITY, 0.0f};
        v = warp_merge(v, a.c2, kMaxCluster);
      }
      if (lane == 0) {
        const RowResult r =
            MODE == kDistill
                ? finish_row<MODE>(a, v, s.in[0], s.t, 0.0f, 0.0f, 0.0f, 0.0f)
                : finish_row<MODE>(a, v, s.in[0], s.t, s.z[0], s.in[1], s.in[2], s.in[3]);
        if (kGrad) {
          s.soft = r.soft;
          s.top = r.top;
          s.scale = r.scale;
        }
        mbar_arrive(smem_u32(&sh.go[b]));
        if (!kGrad) mbar_arrive(smem_u32(&sh.over[i]));
        if (rank == 0) {
          if (a.row_loss) a.row_loss[row] = r.loss;
          if (a.logp) a.logp[row] = r.logp;
        }
      }
      __syncwarp();
    }
    lost = first + it * step;
  }
  if (lost < a.N && lane == 0) red_min_cluster(smem_u32((const void*)&sh.unfinished), 0, lost);
  __syncwarp();
  cluster_arrive();  // no block leaves while another may still write to it
  cluster_wait();
  if (sh.unfinished != INT_MAX) mark_unfinished(a.row_loss, a.logp, sh.unfinished, a.N);
}

// ---------------------------------------------------------------- launches

template <int DT, int MODE, int NT, int VPT>
cudaError_t launch_short(const TokenLossArgs& a, cudaStream_t s) {
  constexpr int kRows = short_rows_per_block(NT);
  return launch_pdl(short_row_kernel<DT, MODE, NT, VPT>, dim3((a.N + kRows - 1) / kRows),
                    dim3(NT * kRows), 0, s, a);
}

template <int DT, int MODE, bool kGrad, bool kTest = false>
cudaError_t launch_long(const TokenLossArgs& a, int C, cudaStream_t s, LeaveArgs leave = {}) {
  auto kernel = long_row_kernel<DT, MODE, kGrad, kTest>;
  static std::atomic<uint64_t> limit_set{0};
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kRingBytes, limit_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(long_threads(kGrad));
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // clusters of this size that run at once, asked once per device
  static std::atomic<int> resident[64][kMaxCluster + 1];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int n = resident[dev & 63][C].load(std::memory_order_relaxed);
  if (n == 0) {
    cfg.gridDim = dim3(C);
    if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    resident[dev & 63][C].store(n, std::memory_order_relaxed);
  }
  if (kTest && n > kLeaveClusters) n = kLeaveClusters;
  cfg.gridDim = dim3((unsigned)(a.N < n ? a.N : n) * C);
  return cudaLaunchKernelEx(&cfg, kernel, a, leave);
}

// A block's part of a long row: two of 80 KB and less leave room to load ahead (8192 x
// 131072 bf16, by parts of 32, 48, 64 and 85 KB: 3164, 1118, 874 and 904 us at the time).
constexpr int kPartVecs = 5120;
// Two of 96 KB still fit with a chunk ahead.  That is better than one block more where
// clusters of C fill more SMs than those of C + 1 (1 to 5: 152, 152, 138, 144, 140): bf16
// gradients of 6000 x 43000 by one block 161 us, by two 185; losses of 6000 x 98000 by two
// 162, by three 195; 4000 x 196000 by four 217, by five 234; but 6000 x 128000 gradients by
// three 498, by four 444.
constexpr int kLargePartVecs = 6 * kChunkVecs;

// Blocks of a long row of nvec vectors.
int cluster_of(int nvec) {
  int C = (nvec + kPartVecs - 1) / kPartVecs;
  if ((C == 2 || C == 3 || C == 5) && nvec <= (C - 1) * kLargePartVecs) --C;
  // clusters of 6 fill 138 SMs, of 7 and 8 only 105 and 120 (4096 x 262144 bf16: 742 us
  // with 6, 890 with 8): parts of which two just fit the ring come first
  if (C > 6) C = nvec <= 6 * kLargePartVecs ? 6 : kMaxCluster;
  return C;
}
constexpr int kShortVecs = 1024;

// The variant goes by the row's length alone, so that a row's bits do not depend on
// the batch.
template <int DT, int MODE>
cudaError_t launch_mode(const TokenLossArgs& a, cudaStream_t s) {
  const int nvec = a.V / Vec<DT>::kElems;  // at most so many vectors a row
  // 16384 bf16 rows of 8192, policy gradient: 120 us here, 163 in the ring; rows of 16384
  // 225 here, 192 there.  fp32 vectors have half the work: fewer threads with more of them
  // (rows of 4096: 78 us by 128 threads, 96 by 256; bf16 rows of 8192 144 and 120).
  if (nvec <= 128) return launch_short<DT, MODE, 32, 4>(a, s);
  constexpr bool kWide = DT == kF32;
  if (nvec <= 512) return launch_short<DT, MODE, kWide ? 64 : 128, kWide ? 8 : 4>(a, s);
  if (nvec <= kShortVecs) return launch_short<DT, MODE, kWide ? 128 : 256, kWide ? 8 : 4>(a, s);
  const int C = cluster_of(nvec);
  return a.dlogits ? launch_long<DT, MODE, true>(a, C, s) : launch_long<DT, MODE, false>(a, C, s);
}

template <int DT>
cudaError_t launch_dtype(const TokenLossArgs& a, int mode, cudaStream_t s) {
  return mode == kDistill ? launch_mode<DT, kDistill>(a, s) : launch_mode<DT, kPolicy>(a, s);
}

}  // namespace

cudaError_t launch_token_loss(const TokenLossArgs& a, int mode, int dtype, cudaStream_t s) {
  if (dtype == kF32) return launch_dtype<kF32>(a, mode, s);
  if (dtype == kBf16) return launch_dtype<kBf16>(a, mode, s);
  return launch_dtype<kF16>(a, mode, s);
}

int token_loss_cluster(int V, int dtype) {
  const int nvec = V / (dtype == kF32 ? Vec<kF32>::kElems : Vec<kBf16>::kElems);
  return nvec <= kShortVecs ? 0 : cluster_of(nvec);
}

cudaError_t launch_token_loss_leave(const TokenLossArgs& a, const LeaveArgs& leave,
                                    cudaStream_t s) {
  return launch_long<kBf16, kPolicy, true, true>(a, token_loss_cluster(a.V, kBf16), s, leave);
}

}  // namespace moe
