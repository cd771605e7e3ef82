// router_loss.cu -- load balance of the router: per-expert counts, balance loss
// and z loss of router logits x [T][E], and the logits' gradient.
//
// With p_t = softmax(x_t), L_t = log sum exp x_t, sequences s of consecutive
// rows, n_s live rows of s, n = sum_s n_s, c_se = how often the live rows of s
// chose expert e, and f_se = E c_se / (K n_s) (1 when the load is even):
//   balance = cb / n sum_s sum_e f_se sum_{t in s} p_te
//   z       = cz / n sum_t L_t^2
//   dx_te   = p_te (gb cb / n (f_se - sum_j f_sj p_tj) + gz 2 cz / n L_t)
//             + sum_{k: id_tk = e} w_tk (dw_tk - sum_j w_tj dw_tj)
// (the last term is the gradient of the scores w, a softmax over the chosen
// logits).  The counts are constants of the gradient.
//
// Sums run in a fixed order, so equal inputs give equal bits.  Rows are cut into
// chunks; chunk c of sequence s leaves its partial sums in slot c + s (walking
// the rows, each step from one piece to the next raises c or s, so pieces have
// different slots), and a second kernel adds a sequence's slots up in order.
#include "internal.h"
#include "logits.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPerLane = 32;  // E <= 1024
constexpr int kChunkRows = 128;

int num_chunks(int T) { return (T + kChunkRows - 1) / kChunkRows; }

// Workspace: the status word (as the forward's, for moe_nvfp4_read_status), the
// second kernel's ticket, per sequence its share of the losses and the bad-id
// flag, then per slot [E] probability sums, [E] counts, z sum, live rows, bad ids.
struct Ws {
  int32_t* status;
  int32_t* ticket;
  float2* seq;      // [S] balance and z sums
  int32_t* seq_bad; // [S]
  float* slot;      // [slots][2 E + 3]
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
Ws carve(void* ws, int S) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Ws w;
  w.status = reinterpret_cast<int32_t*>(p);
  w.ticket = w.status + kStatusWords;
  w.seq = reinterpret_cast<float2*>(p + 256);
  w.seq_bad = reinterpret_cast<int32_t*>(p + 256 + up256((size_t)S * sizeof(float2)));
  w.slot = reinterpret_cast<float*>(p + 256 + up256((size_t)S * sizeof(float2)) +
                                    up256((size_t)S * sizeof(int32_t)));
  return w;
}

// Sequence of a row: the last s with offsets[s] <= row, or -1 outside all sequences.
__device__ __forceinline__ int sequence_of(const int32_t* off, int S, int row) {
  if (!off) return 0;
  if (row < off[0] || row >= off[S]) return -1;
  int lo = 0, hi = S;  // off[lo] <= row < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One router row in a warp's registers: lane + 32 i holds expert lane + 32 i.
template <int DT>
struct Row {
  float p[kMaxPerLane];  // softmax, 0 beyond E
  float m, r;            // the largest logit (0 if none is finite) and 1 / sum (0 then)
  float lse;             // 0 for a row without a finite logit
  __device__ __forceinline__ void load(const typename LogitType<DT>::type* x, int E, int lane) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
      if (32 * i >= E) break;
      const int e = lane + 32 * i;
      p[i] = e < E ? load_logit<DT>(x + e) : -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = finite_ref(warp_max(m));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
      if (32 * i >= E) break;
      p[i] = ex2((p[i] - m) * kLog2e);
      s += p[i];
    }
    s = warp_sum(s);
    lse = s == 0.0f ? 0.0f : m + logf(s);
    r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
      if (32 * i >= E) break;
      p[i] *= r;
    }
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads) router_partial_kernel(const RouterLossArgs a, Ws w) {
  using L = typename LogitType<DT>::type;
  extern __shared__ float s_p[];  // [kWarps][E], then int[E]
  int* s_hist = reinterpret_cast<int*>(s_p + kWarps * a.E);
  __shared__ float s_z[kWarps];
  __shared__ int s_n[kWarps], s_bad[kWarps];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && tid == 0) *w.ticket = 0;
  const int row_end = min(a.T, (int)(blockIdx.x + 1) * kChunkRows);
  int row0 = blockIdx.x * kChunkRows;
  for (int e = tid; e < a.E; e += kThreads) s_hist[e] = 0;
  __syncthreads();
  while (row0 < row_end) {  // one piece: the rows of one sequence in this chunk
    const int s = sequence_of(a.offsets, a.S, row0);
    if (s < 0) {  // before the first sequence or past the last
      row0 = row0 < a.offsets[0] ? min(row_end, a.offsets[0]) : row_end;
      continue;
    }
    const int row1 = a.offsets ? min(row_end, a.offsets[s + 1]) : row_end;
    float acc[kMaxPerLane];
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0, bad = 0;
    for (int t = row0 + warp; t < row1; t += kWarps) {
      if (a.mask && !a.mask[t]) continue;
      Row<DT> r;
      r.load(static_cast<const L*>(a.logits) + t * a.ld, a.E, lane);
#pragma unroll
      for (int i = 0; i < kMaxPerLane; ++i) {
        if (32 * i >= a.E) break;
        acc[i] += r.p[i];
      }
      z += r.lse * r.lse;
      ++n;
      if (lane < a.K) {
        const int64_t at = (int64_t)t * a.K + lane;
        const int id = load_id(a.ids, a.ids64, at);
        if (id >= 0 && id < a.E) atomicAdd(&s_hist[id], 1);
        const bool empty = a.ids64 ? static_cast<const long long*>(a.ids)[at] == -1 : id == -1;
        bad |= !(id >= 0 && id < a.E) && !empty;
      }
    }
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) s_p[warp * a.E + e] = acc[i];
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      s_z[warp] = z;
      s_n[warp] = n;
      s_bad[warp] = bad;
    }
    __syncthreads();
    float* slot = w.slot + (size_t)(blockIdx.x + s) * (2 * a.E + 3);
    for (int e = tid; e < a.E; e += kThreads) {
      float sum = 0.0f;
      for (int i = 0; i < kWarps; ++i) sum += s_p[i * a.E + e];
      slot[e] = sum;
      slot[a.E + e] = __int_as_float(s_hist[e]);
      s_hist[e] = 0;
    }
    if (tid == 0) {
      float zs = 0.0f;
      int ns = 0, bs = 0;
      for (int i = 0; i < kWarps; ++i) {
        zs += s_z[i];
        ns += s_n[i];
        bs |= s_bad[i];
      }
      slot[2 * a.E] = zs;
      slot[2 * a.E + 1] = __int_as_float(ns);
      slot[2 * a.E + 2] = __int_as_float(bs);
    }
    __syncthreads();
    row0 = max(row1, row0 + 1);
  }
}

__global__ void __launch_bounds__(kThreads) router_combine_kernel(const RouterLossArgs a, Ws w,
                                                                  int chunks) {
  __shared__ float s_a[kThreads], s_b[kThreads];
  __shared__ int s_i[kThreads];
  __shared__ int s_last;
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, tid = threadIdx.x;
  const int r0 = a.offsets ? a.offsets[s] : 0, r1 = a.offsets ? a.offsets[s + 1] : a.T;
  int c0 = max(0, r0) / kChunkRows, c1 = (min(r1, a.T) + kChunkRows - 1) / kChunkRows;
  if (r1 <= r0) c1 = c0;
  float z = 0.0f;
  int n = 0, bad = 0;
  for (int c = c0; c < c1; ++c) {
    const float* slot = w.slot + (size_t)(c + s) * (2 * a.E + 3);
    z += slot[2 * a.E];
    n += __float_as_int(slot[2 * a.E + 1]);
    bad |= __float_as_int(slot[2 * a.E + 2]);
  }
  float dot = 0.0f;
  for (int e = tid; e < a.E; e += kThreads) {
    float p = 0.0f;
    int cnt = 0;
    for (int c = c0; c < c1; ++c) {
      const float* slot = w.slot + (size_t)(c + s) * (2 * a.E + 3);
      p += slot[e];
      cnt += __float_as_int(slot[a.E + e]);
    }
    a.counts[(size_t)s * a.E + e] = cnt;
    dot += (float)cnt * p;
  }
  s_a[tid] = dot;
  __syncthreads();
  if (tid == 0) {
    float sum = 0.0f;
    for (int i = 0; i < kThreads; ++i) sum += s_a[i];
    const float f = n > 0 ? (float)a.E / ((float)a.K * (float)n) : 0.0f;
    w.seq[s] = make_float2(n > 0 ? f * sum : 0.0f, z);
    w.seq_bad[s] = bad;
    a.tokens[s] = n;
    s_last = atom_add_acq_rel_gpu(w.ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // the last block adds the sequences up
  float bal = 0.0f, zs = 0.0f;
  int total = 0;
  bad = 0;
  for (int i = tid; i < a.S; i += kThreads) {
    const float2 v = __ldcg(&w.seq[i]);
    bal += v.x;
    zs += v.y;
    total += __ldcg(&a.tokens[i]);
    bad |= __ldcg(&w.seq_bad[i]);
  }
  s_a[tid] = bal;
  s_b[tid] = zs;
  s_i[tid] = total;
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    bal = zs = 0.0f;
    total = 0;
    for (int i = 0; i < kThreads; ++i) {
      bal += s_a[i];
      zs += s_b[i];
      total += s_i[i];
    }
    const float per = total > 0 ? 1.0f / (float)total : 0.0f;
    a.losses[0] = total > 0 ? a.balance_coef * bal * per : 0.0f;
    a.losses[1] = total > 0 ? a.z_coef * zs * per : 0.0f;
    a.tokens[a.S] = total;
    *w.status = bad ? kFlagBadExpertId : 0;
  }
}

// One warp per row.
template <int DT>
__global__ void __launch_bounds__(kThreads) router_grad_kernel(const RouterLossArgs a) {
  using L = typename LogitType<DT>::type;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const L* x = static_cast<const L*>(a.logits) + t * a.ld;
  L* dx = static_cast<L*>(a.dlogits) + t * a.ld_grad;
  const int s = sequence_of(a.offsets, a.S, t);
  if (s < 0 || (a.mask && !a.mask[t])) {
    for (int e = lane; e < a.E; e += 32) store_logit<DT>(dx + e, 0.0f);
    return;
  }
  // the scores' gradient at this lane's slot; slots that repeat an expert add up
  int id = -1;
  float v = 0.0f, xid = 0.0f;
  if (a.topk_w) {
    float wk = 0.0f, dwk = 0.0f;
    if (lane < a.K) {
      id = load_id(a.ids, a.ids64, (int64_t)t * a.K + lane);
      if (id >= a.E) id = -1;
      if (id >= 0) {
        wk = a.topk_w[(int64_t)t * a.K + lane];
        dwk = a.d_topk_w[(int64_t)t * a.K + lane];
        xid = load_logit<DT>(x + id);
      }
    }
    const float mine = wk * (dwk - warp_sum(wk * dwk));
    for (int k = 0; k < a.K; ++k) {
      const float o = __shfl_sync(0xFFFFFFFFu, mine, k);
      v += __shfl_sync(0xFFFFFFFFu, id, k) == id ? o : 0.0f;
    }
  }
  Row<DT> r;
  r.load(x, a.E, lane);
  const int n_s = a.tokens[s], n = a.tokens[a.S];
  const float per = n > 0 ? 1.0f / (float)n : 0.0f;
  const float f1 = n_s > 0 ? (float)a.E / ((float)a.K * (float)n_s) : 0.0f;
  const float gb = (a.loss_grad ? a.loss_grad[0] : 1.0f) * a.balance_coef * per;
  const float gz = (a.loss_grad ? a.loss_grad[1] : 1.0f) * 2.0f * a.z_coef * per;
  const int32_t* cnt = a.counts + (size_t)s * a.E;
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    if (32 * i >= a.E) break;
    const int e = lane + 32 * i;
    if (e < a.E) dot += (float)cnt[e] * f1 * r.p[i];
  }
  dot = warp_sum(dot);
  const float add = gz * r.lse;
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    if (32 * i >= a.E) break;
    const int e = lane + 32 * i;
    if (e < a.E) store_logit<DT>(dx + e, r.p[i] * (gb * ((float)cnt[e] * f1 - dot) + add));
  }
  if (a.topk_w) {
    __syncwarp();  // the chosen experts' entries overwrite what the loop stored
    if (id >= 0) {
      const float p = ex2((xid - r.m) * kLog2e) * r.r;
      store_logit<DT>(dx + id, p * (gb * ((float)cnt[id] * f1 - dot) + add) + v);
    }
  }
}

template <int DT>
cudaError_t launch_partial(const RouterLossArgs& a, const Ws& w, cudaStream_t s) {
  const int smem = (kWarps + 1) * a.E * (int)sizeof(float);  // at most 36 KB
  return launch_pdl(router_partial_kernel<DT>, dim3(num_chunks(a.T)), dim3(kThreads), smem, s, a, w);
}

}  // namespace

size_t router_loss_ws_bytes(int T, int E, int S) {
  return 256 + up256((size_t)S * sizeof(float2)) + up256((size_t)S * sizeof(int32_t)) +
         ((size_t)num_chunks(T) + S) * (2 * (size_t)E + 3) * sizeof(float);
}

cudaError_t launch_router_loss(const RouterLossArgs& a, int dtype, cudaStream_t s) {
  const Ws w = carve(a.ws, a.S);
  const cudaError_t e = dtype == kF32    ? launch_partial<kF32>(a, w, s)
                        : dtype == kBf16 ? launch_partial<kBf16>(a, w, s)
                                         : launch_partial<kF16>(a, w, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(router_combine_kernel, dim3(a.S), dim3(kThreads), 0, s, a, w, num_chunks(a.T));
}

cudaError_t launch_router_loss_grad(const RouterLossArgs& a, int dtype, cudaStream_t s) {
  const dim3 grid((a.T + kWarps - 1) / kWarps), block(kThreads);
  if (dtype == kF32) return launch_pdl(router_grad_kernel<kF32>, grid, block, 0, s, a);
  if (dtype == kBf16) return launch_pdl(router_grad_kernel<kBf16>, grid, block, 0, s, a);
  return launch_pdl(router_grad_kernel<kF16>, grid, block, 0, s, a);
}

}  // namespace moe
