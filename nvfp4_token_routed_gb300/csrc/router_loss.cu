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
// A row lies in the registers of 8, 16 or 32 lanes, 32 values a lane at most, with the
// next row's loads in flight: the fewer lanes, the fewer instructions a row (a warp's
// shuffles, logarithms and score slots serve 4 or 2 rows at once).  Sums run in a fixed order, so equal inputs give equal bits: rows are cut into chunks, one a
// block; chunk c of sequence s leaves its partial sums in slot c + s (walking the
// rows, each step from one piece to the next raises c or s, so pieces have different
// slots), and a second kernel adds a sequence's slots up in order, its last block the
// sequences.  Small batches take one block and one launch.
#include <type_traits>

#include "internal.h"
#include "logits.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;        // of a block of many
constexpr int kSmallWarps = 16;  // of the only block of a small batch
constexpr int kSmallRows = 128;  // the largest small batch
constexpr int kSmallSeqs = 4;
constexpr int kMaxBlocks = 152 * 4;

// Rows of a chunk: a block's warps share them; more rows a block than warps only where
// `blocks` blocks fill the device.
int chunk_rows(int T, int blocks) {
  const int r = (T + blocks - 1) / blocks;
  return (r + kWarps - 1) / kWarps * kWarps;
}
// At least the chunks of this and of any smaller batch.
int max_chunks(int T) {
  const int c = (T + kWarps - 1) / kWarps;
  return c < kMaxBlocks ? c : kMaxBlocks;
}

// Workspace: the status word (as the forward's, for moe_nvfp4_read_status), the
// second kernel's ticket, per sequence its z sum and bad-id flag, per sequence and
// 32 experts the sum of counts times probabilities, then per slot [E] probability
// sums, [E] counts, z sum, live rows, bad ids.
struct Ws {
  int32_t* status;
  int32_t* ticket;
  float2* seq;
  float* dots;
  float* slot;
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int expert_blocks(int E) { return (E + 31) / 32; }
size_t seq_bytes(int S) { return up256((size_t)S * sizeof(float2)); }
size_t dots_bytes(int S, int E) { return up256((size_t)S * expert_blocks(E) * sizeof(float)); }
Ws carve(void* ws, int E, int S) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Ws w;
  w.status = reinterpret_cast<int32_t*>(p);
  w.ticket = w.status + kStatusWords;
  w.seq = reinterpret_cast<float2*>(p + 256);
  w.dots = reinterpret_cast<float*>(p + 256 + seq_bytes(S));
  w.slot = reinterpret_cast<float*>(p + 256 + seq_bytes(S) + dots_bytes(S, E));
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

// How NL lanes hold a row: NV vectors of 16 bytes a lane, vector i of lane l at column
// (NL i + l) W.  Rows that do not start on 16-byte boundaries, or whose length is no
// multiple of W, are read and written by the element, with the same columns in the same
// lanes and so the same bits.
template <int DT, int NL, int NV>
struct Raw {
  using L = typename LogitType<DT>::type;
  using V = Vec<DT>;
  static constexpr int W = V::kElems;
  static constexpr int kN = W * NV;
  V v[NV];
  static __device__ __forceinline__ int column(int n, int l) {
    return (n / W * NL + l) * W + n % W;
  }
  __device__ __forceinline__ void load(const L* row, int E, int l, bool aligned) {
    if (aligned) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (NL * i + l) * W;
        if (c < E) v[i].v = *reinterpret_cast<const uint4*>(row + c);
        else v[i].fill(V::kNegInf);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (NL * i + l) * W;
      L x[W];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (DT == kF32) x[j] = c + j < E ? row[c + j] : -INFINITY;
        else x[j] = c + j < E ? row[c + j] : (L)(V::kNegInf >> 16);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == kF32) v[i].set_word(j, __float_as_uint(x[j]));
        else v[i].set_word(j, (uint32_t)x[2 * j] | (uint32_t)x[2 * j + 1] << 16);
      }
    }
  }
  __device__ __forceinline__ void fill() {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i].fill(V::kNegInf);
  }
  __device__ __forceinline__ void get(float (&f)[kN]) const {
#pragma unroll
    for (int n = 0; n < kN; n += 2) {
      const float2 p = unpack2(pack2(v[n / W].pair(n % W / 2)));
      f[n] = p.x;
      f[n + 1] = p.y;
    }
  }
  static __device__ __forceinline__ void store(L* row, int E, int l, bool aligned,
                                               const float (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (NL * i + l) * W;
      if (aligned) {
        V g;
#pragma unroll
        for (int j = 0; j < V::kPairs; ++j)
          g.set_pair(j, make_float2(f[i * W + 2 * j], f[i * W + 2 * j + 1]));
        if (c < E) *reinterpret_cast<uint4*>(row + c) = g.v;
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (c + j < E) store_logit<DT>(row + c + j, f[i * W + j]);
      }
    }
  }
};

// Sum and maximum over the NL lanes of a row.
template <int NL>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = NL / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}
template <int NL>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int off = NL / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

// The row's softmax over its lanes: e = 2^((x - m) log2 e), p = e r; a row without a
// finite logit has p = 0 and lse = 0.
struct RowStats {
  float m, r, lse;
};
template <int NL, int N>
__device__ __forceinline__ RowStats exponentials(float (&p)[N]) {
  float m = p[0];
#pragma unroll
  for (int n = 1; n < N; ++n) m = fmaxf(m, p[n]);
  m = finite_ref(row_max<NL>(m));
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    p[n] = ex2((p[n] - m) * kLog2e);
    s[n & 1] += p[n];
  }
  const float sum = row_sum<NL>(s[0] + s[1]);
  RowStats st;
  st.m = m;
  st.lse = sum == 0.0f ? 0.0f : m + logf(sum);
  st.r = sum == 0.0f ? 0.0f : 1.0f / sum;
  return st;
}

// One piece: the sums over the live rows of [row0, row1) by a block of NW warps.
// Afterwards, for all threads: sum of the warps' s_p[w][e] is the probability sum,
// s_hist the counts; z, n and bad are thread 0's.
struct PieceScalars {
  float z;
  int n, bad;
};
template <int DT, int NL, int NV, int NW>
__device__ __forceinline__ PieceScalars piece_sums(const RouterLossArgs& a, int row0, int row1,
                                                   float* s_p, int* s_hist) {
  using R = Raw<DT, NL, NV>;
  constexpr int kRows = 32 / NL * NW;  // rows at a time
  __shared__ float s_z[NW];
  __shared__ int s_n[NW], s_bad[NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % NL;
  for (int e = tid; e < a.E; e += NW * 32) s_hist[e] = 0;
  __syncthreads();
  float acc[R::kN];
#pragma unroll
  for (int i = 0; i < R::kN; ++i) acc[i] = 0.0f;
  float z = 0.0f;
  int n = 0, bad = 0;
  const auto* base = static_cast<const typename R::L*>(a.logits);
  // the lane's slot of row t; an id below -1 or from E on is bad, 64-bit ids beyond 32
  // bits read as -2
  auto fetch = [&](int t, R& row, int& id) {
    const bool live = t < row1 && (!a.mask || a.mask[t]);
    id = -1;
    if (!live) return false;
    row.load(base + t * a.ld, a.E, l, a.aligned);
    if (l < a.K) {
      const int64_t at = (int64_t)t * a.K + l;
      if (!a.ids64) {
        id = static_cast<const int32_t*>(a.ids)[at];
      } else {
        const long long v = static_cast<const long long*>(a.ids)[at];
        id = v < -1 || v > INT32_MAX ? -2 : (int)v;
      }
    }
    return true;
  };
  const int trips = (row1 - row0 + kRows - 1) / kRows;
  int t = row0 + tid / NL;
  R next;
  next.fill();
  int next_id;
  bool next_live = fetch(t, next, next_id);
  for (int i = 0; i < trips; ++i, t += kRows) {
    const R row = next;
    const int id = next_id;
    const bool live = next_live;
    next_live = fetch(t + kRows, next, next_id);
    if (!__any_sync(0xFFFFFFFFu, live)) continue;
    float p[R::kN];
    row.get(p);
    const RowStats st = exponentials<NL>(p);
    const float r = live ? st.r : 0.0f;
    if (live) {
#pragma unroll
      for (int i = 0; i < R::kN; ++i) acc[i] += p[i] * r;
      z += st.lse * st.lse;
      ++n;
    }
    if (id >= 0 && id < a.E) atomicAdd(&s_hist[id], 1);
    else if (id != -1) bad = 1;
  }
  // the warp's rows: lanes NL apart hold the same columns
#pragma unroll
  for (int off = NL; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < R::kN; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
    z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
  }
  if (lane < NL) {
#pragma unroll
    for (int i = 0; i < R::kN; ++i) {
      const int e = R::column(i, l);
      if (e < a.E) s_p[warp * a.E + e] = acc[i];
    }
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
    s_bad[warp] = bad;
  }
  __syncthreads();
  PieceScalars r = {0.0f, 0, 0};
  if (tid == 0) {
    for (int i = 0; i < NW; ++i) {
      r.z += s_z[i];
      r.n += s_n[i];
      r.bad |= s_bad[i];
    }
  }
  return r;
}
template <int NW>
__device__ __forceinline__ float warps_sum(const float* s_p, int E, int e) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) sum += s_p[i * E + e];
  return sum;
}

template <int DT, int NL, int NV>
__global__ void __launch_bounds__(kWarps * 32, 2) router_partial_kernel(const RouterLossArgs a, Ws w,
                                                                     int rows) {
  extern __shared__ float s_p[];  // [kWarps][E], then int[E]
  int* s_hist = reinterpret_cast<int*>(s_p + kWarps * a.E);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && tid == 0) *w.ticket = 0;
  const int row_end = (int)min((int64_t)a.T, ((int64_t)blockIdx.x + 1) * rows);
  int row0 = blockIdx.x * rows;
  while (row0 < row_end) {  // one piece: the rows of one sequence in this chunk
    const int s = sequence_of(a.offsets, a.S, row0);
    if (s < 0) {  // before the first sequence or past the last
      row0 = row0 < a.offsets[0] ? min(row_end, a.offsets[0]) : row_end;
      continue;
    }
    const int row1 = a.offsets ? min(row_end, a.offsets[s + 1]) : row_end;
    const PieceScalars r = piece_sums<DT, NL, NV, kWarps>(a, row0, row1, s_p, s_hist);
    float* slot = w.slot + (size_t)(blockIdx.x + s) * (2 * a.E + 3);
    for (int e = tid; e < a.E; e += kWarps * 32) {
      slot[e] = warps_sum<kWarps>(s_p, a.E, e);
      slot[a.E + e] = __int_as_float(s_hist[e]);
    }
    if (tid == 0) {
      slot[2 * a.E] = r.z;
      slot[2 * a.E + 1] = __int_as_float(r.n);
      slot[2 * a.E + 2] = __int_as_float(r.bad);
    }
    __syncthreads();
    row0 = max(row1, row0 + 1);
  }
}

// The two losses from the sums, and what goes with them.
__device__ __forceinline__ void write_losses(const RouterLossArgs& a, const Ws& w, float bal,
                                             float z, int n, int bad) {
  const float per = n > 0 ? 1.0f / (float)n : 0.0f;
  a.losses[0] = n > 0 ? a.balance_coef * bal * per : 0.0f;
  // a row of the lowest logits has a square beyond fp32: not 0 * inf where the term is off
  a.losses[1] = n > 0 && !(a.z_coef == 0.0f && isinf(z)) ? a.z_coef * z * per : 0.0f;
  a.tokens[a.S] = n;
  *w.status = bad ? kFlagBadExpertId : 0;
}
__device__ __forceinline__ float even_share(const RouterLossArgs& a, int n_s) {
  return n_s > 0 ? (float)a.E / ((float)a.K * (float)n_s) : 0.0f;
}

// Block (s, j): sequence s, groups j, j + gridDim.y, ... of 32 experts along x, the
// sequence's slots along y.
__global__ void __launch_bounds__(1024) router_combine_kernel(const RouterLossArgs a, Ws w,
                                                              int rows) {
  __shared__ float s_a[1024], s_b[1024];
  __shared__ int s_i[1024];
  __shared__ int s_last;
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, lane = threadIdx.x, y = threadIdx.y, Y = blockDim.y;
  const int tid = y * 32 + lane, threads = Y * 32;
  const int r0 = a.offsets ? max(0, a.offsets[s]) : 0;
  const int r1 = a.offsets ? min(a.T, a.offsets[s + 1]) : a.T;
  const int c0 = r0 / rows, c1 = r1 > r0 ? (r1 + rows - 1) / rows : c0;
  const size_t stride = 2 * (size_t)a.E + 3;
  float z = 0.0f, dots = 0.0f;
  int n = 0, bad = 0;
  for (int e = blockIdx.y * 32 + lane; e - lane < a.E; e += gridDim.y * 32) {
    float p = 0.0f;
    int cnt = 0;
    const bool meta = blockIdx.y == 0 && e == 0;
#pragma unroll 8
    for (int c = c0 + y; c < c1; c += Y) {
      const float* slot = w.slot + (size_t)(c + s) * stride;
      if (e < a.E) {
        p += slot[e];
        cnt += __float_as_int(slot[a.E + e]);
      }
      if (meta) {
        z += slot[2 * a.E];
        n += __float_as_int(slot[2 * a.E + 1]);
        bad |= __float_as_int(slot[2 * a.E + 2]);
      }
    }
    __syncthreads();  // the sums below of the group before
    s_a[tid] = p;
    s_i[tid] = cnt;
    __syncthreads();
    for (int half = Y / 2; half > 0; half >>= 1) {
      if (y < half) {
        s_a[tid] += s_a[tid + half * 32];
        s_i[tid] += s_i[tid + half * 32];
      }
      __syncthreads();
    }
    if (y == 0 && e < a.E) {
      a.counts[(size_t)s * a.E + e] = s_i[lane];
      dots += (float)s_i[lane] * s_a[lane];
    }
  }
  if (y == 0) {
    dots = warp_sum(dots);
    if (lane == 0) w.dots[(size_t)s * gridDim.y + blockIdx.y] = dots;
  }
  __syncthreads();
  if (blockIdx.y == 0) {
    if (lane == 0) {
      s_a[y] = z;
      s_i[y] = n;
      s_i[32 + y] = bad;
    }
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < Y; ++i) {
        z += s_a[i];
        n += s_i[i];
        bad |= s_i[32 + i];
      }
      w.seq[s] = make_float2(z, __int_as_float(bad));
      a.tokens[s] = n;
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0)
    s_last = atom_add_acq_rel_gpu(w.ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
  __syncthreads();
  if (!s_last) return;
  // the last block adds the sequences up
  float bal = 0.0f;
  z = 0.0f;
  n = bad = 0;
  const int eb = gridDim.y;
#pragma unroll 4
  for (int i = tid; i < a.S * eb; i += threads) {
    const int n_s = __ldcg(&a.tokens[i / eb]);
    const float dot = __ldcg(&w.dots[i]);
    bal += n_s > 0 ? even_share(a, n_s) * dot : 0.0f;
  }
#pragma unroll 4
  for (int i = tid; i < a.S; i += threads) {
    const float2 v = __ldcg(&w.seq[i]);
    z += v.x;
    bad |= __float_as_int(v.y);
    n += __ldcg(&a.tokens[i]);
  }
  const int any_bad = __syncthreads_or(bad);
  s_a[tid] = bal;
  s_b[tid] = z;
  s_i[tid] = n;
  __syncthreads();
  for (int half = threads / 2; half > 0; half >>= 1) {
    if (tid < half) {
      s_a[tid] += s_a[tid + half];
      s_b[tid] += s_b[tid + half];
      s_i[tid] += s_i[tid + half];
    }
    __syncthreads();
  }
  if (tid == 0) write_losses(a, w, s_a[0], s_b[0], s_i[0], any_bad);
}

// A small batch: one block, the sequences one after another.
template <int DT, int NV>
__global__ void __launch_bounds__(kSmallWarps * 32) router_small_kernel(const RouterLossArgs a,
                                                                        Ws w) {
  extern __shared__ float s_p[];  // [kSmallWarps][E], then int[E]
  int* s_hist = reinterpret_cast<int*>(s_p + kSmallWarps * a.E);
  __shared__ float s_dot[kSmallWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float bal = 0.0f, z = 0.0f;
  int n = 0, bad = 0;
  for (int s = 0; s < a.S; ++s) {
    const int r0 = a.offsets ? max(0, a.offsets[s]) : 0;
    const int r1 = a.offsets ? min(a.T, a.offsets[s + 1]) : a.T;
    const PieceScalars r = piece_sums<DT, 32, NV, kSmallWarps>(a, r0, r1, s_p, s_hist);
    float dot = 0.0f;
    for (int e = tid; e < a.E; e += kSmallWarps * 32) {
      const int cnt = s_hist[e];
      a.counts[(size_t)s * a.E + e] = cnt;
      dot += (float)cnt * warps_sum<kSmallWarps>(s_p, a.E, e);
    }
    dot = warp_sum(dot);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (tid == 0) {
      dot = 0.0f;
      for (int i = 0; i < kSmallWarps; ++i) dot += s_dot[i];
      if (r.n > 0) bal += even_share(a, r.n) * dot;
      a.tokens[s] = r.n;
      z += r.z;
      n += r.n;
      bad |= r.bad;
    }
  }
  if (tid == 0) write_losses(a, w, bal, z, n, bad);
}

// NL lanes for `rows` rows, 32 / NL apart; f_se stays in registers while the sequence does.
template <int DT, int NL, int NV>
__global__ void __launch_bounds__(kWarps * 32, 2) router_grad_kernel(const RouterLossArgs a,
                                                                  int rows) {
  using R = Raw<DT, NL, NV>;
  using L = typename LogitType<DT>::type;
  constexpr int kSub = 32 / NL;  // rows of a warp at a time
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, l = lane % NL;
  const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * rows * kSub;
  const L* x = static_cast<const L*>(a.logits);
  L* dx = static_cast<L*>(a.dlogits);
  const int n = a.tokens[a.S];
  const float per = n > 0 ? 1.0f / (float)n : 0.0f;
  const float gb = (a.loss_grad ? a.loss_grad[0] : 1.0f) * a.balance_coef * per;
  const float gz = (a.loss_grad ? a.loss_grad[1] : 1.0f) * 2.0f * a.z_coef * per;
  int s = -1, s_end = 0;  // sequence of the rows before s_end
  float f1 = 0.0f, f[R::kN];
#pragma unroll
  for (int i = 0; i < R::kN; ++i) f[i] = 0.0f;
  // a row and this lane's slot of its scores
  struct Slot {
    int id;
    float w, dw;
  };
  auto fetch = [&](int64_t t, R& row, Slot& k) {
    k = {-1, 0.0f, 0.0f};
    if (t >= a.T || (a.mask && !a.mask[t])) return false;
    row.load(x + t * a.ld, a.E, l, a.aligned);
    if (a.topk_w && l < a.K) {
      const int64_t at = t * a.K + l;
      const int id = load_id(a.ids, a.ids64, at);
      if (id >= 0 && id < a.E) k = {id, a.topk_w[at], a.d_topk_w[at]};
    }
    return true;
  };
  R next;
  next.fill();
  Slot next_slot;
  int64_t t = first + lane / NL;
  bool next_live = fetch(t, next, next_slot);
  for (int step = 0; step < rows; ++step, t += kSub) {
    const R row = next;
    const Slot slot = next_slot;
    bool live = next_live;
    next_live = step + 1 < rows && fetch(t + kSub, next, next_slot);
    if (live && (t >= s_end || s < 0)) {
      s = sequence_of(a.offsets, a.S, (int)t);
      if (s >= 0) {
        s_end = a.offsets ? a.offsets[s + 1] : a.T;
        f1 = even_share(a, a.tokens[s]);
        const int32_t* cnt = a.counts + (size_t)s * a.E;
#pragma unroll
        for (int i = 0; i < R::kN; i += 4) {
          const int e = R::column(i, l);  // four columns in a row
          if (a.counts_aligned) {
            const int4 c = e < a.E ? *reinterpret_cast<const int4*>(cnt + e) : int4{0, 0, 0, 0};
            f[i] = (float)c.x * f1;
            f[i + 1] = (float)c.y * f1;
            f[i + 2] = (float)c.z * f1;
            f[i + 3] = (float)c.w * f1;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[i + j] = e + j < a.E ? (float)cnt[e + j] * f1 : 0.0f;
          }
        }
      }
    }
    live = live && s >= 0;
    // the chosen experts' entries
    int id = live ? slot.id : -1;
    float v = 0.0f, x_id = 0.0f, f_id = 0.0f;
    if (a.topk_w) {
      if (id >= 0) {
        x_id = load_logit<DT>(x + t * a.ld + id);
        f_id = (float)a.counts[(size_t)s * a.E + id] * f1;
      }
      const float mean = row_sum<NL>(id >= 0 ? slot.w * slot.dw : 0.0f);
      const float mine = id >= 0 ? slot.w * (slot.dw - mean) : 0.0f;
      v = mine;
      // slots that repeat an expert add up, in the order of the slots
      const uint32_t key = id >= 0 ? (uint32_t)(lane / NL) << 16 | id : 0x80000000u | lane;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, key);
      if (__any_sync(0xFFFFFFFFu, (same & (same - 1)) != 0)) {
        v = 0.0f;
        for (int k = 0; k < 32; ++k) {
          const float o = __shfl_sync(0xFFFFFFFFu, mine, k);
          v += (same >> k) & 1 ? o : 0.0f;
        }
      }
    }
    float p[R::kN];
    row.get(p);
    const RowStats st = exponentials<NL>(p);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < R::kN; ++i) dot += f[i] * p[i];
    dot = row_sum<NL>(dot) * st.r;
    const float add = gz * st.lse - gb * dot, r = live ? st.r : 0.0f;
    const float c1 = gb * r, c0 = add * r;
#pragma unroll
    for (int i = 0; i < R::kN; ++i) p[i] = live ? p[i] * fmaf(c1, f[i], c0) : 0.0f;
    __syncwarp();  // in place, x_id was read before the lanes overwrite the row
    if (t < a.T) R::store(dx + t * a.ld_grad, a.E, l, a.aligned, p);
    if (a.topk_w) {
      __syncwarp();  // the entries overwrite what the lanes stored
      if (id >= 0)
        store_logit<DT>(dx + t * a.ld_grad + id,
                        ex2((x_id - st.m) * kLog2e) * fmaf(c1, f_id, c0) + v);
    }
  }
}

// fn(lanes a row, vectors a lane).  With 32 lanes a small batch has the lowest latency
// and short sequences the least to reload; otherwise the fewest lanes that hold the row
// at 32 values each: 65536 rows of 256 bf16 logits and 61 sequences, loss and gradient,
// take 47 us with 8 lanes and 65 us with 32; 20000 rows in 300 sequences 60 and 45 us.
constexpr int kManyRows = 4096, kLongSequence = 512;
template <int V>
using Int = std::integral_constant<int, V>;
template <int DT, typename F>
cudaError_t with_layout(const RouterLossArgs& a, F fn) {
  constexpr int W = Vec<DT>::kElems;
  const int nv = (a.E + W - 1) / W;  // vectors a row
  const bool many = a.T >= kManyRows && a.T / a.S >= kLongSequence;
  if (many && a.K <= 8) {
    if (nv <= 8) return fn(Int<8>{}, Int<1>{});
    if (nv <= 16) return fn(Int<8>{}, Int<2>{});
    if (nv <= 32) return fn(Int<8>{}, Int<4>{});
  }
  if (many && a.K <= 16) {
    if constexpr (DT == kF32) {
      if (nv > 32 && nv <= 64) return fn(Int<16>{}, Int<4>{});
      if (nv > 64 && nv <= 96) return fn(Int<16>{}, Int<6>{});
      if (nv > 64 && nv <= 128) return fn(Int<16>{}, Int<8>{});
    } else {
      if (nv > 32 && nv <= 48) return fn(Int<16>{}, Int<3>{});
      if (nv > 32 && nv <= 64) return fn(Int<16>{}, Int<4>{});
    }
  }
  if (nv <= 32) return fn(Int<32>{}, Int<1>{});
  if (nv <= 64) return fn(Int<32>{}, Int<2>{});
  if constexpr (DT == kF32) {
    if (nv <= 96) return fn(Int<32>{}, Int<3>{});
    if (nv > 128) return fn(Int<32>{}, Int<8>{});
  }
  return fn(Int<32>{}, Int<4>{});
}
template <int DT>
bool rows_aligned(const RouterLossArgs& a) {
  auto ok = [](const void* p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (DT == kF32 ? 4 : 2) % 16 == 0);
  };
  return a.E % Vec<DT>::kElems == 0 && ok(a.logits, a.ld) && ok(a.dlogits, a.ld_grad);
}

template <int DT>
cudaError_t launch_loss(RouterLossArgs a, cudaStream_t s) {
  const Ws w = carve(a.ws, a.E, a.S);
  a.aligned = rows_aligned<DT>(a);
  return with_layout<DT>(a, [&](auto nl, auto nv) {
    constexpr int kNL = decltype(nl)::value, kNV = decltype(nv)::value;
    if constexpr (kNL == 32) {
      if (a.T <= kSmallRows && a.S <= kSmallSeqs) {
        auto kernel = router_small_kernel<DT, kNV>;
        static std::atomic<uint64_t> limit_set{0};
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel),
                                                (kSmallWarps + 1) * 1024 * 4, limit_set);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(1), dim3(kSmallWarps * 32), (kSmallWarps + 1) * a.E * 4, s,
                          a, w);
      }
    }
    // two blocks of the wide layouts fit an SM, and each has its sums to write
    const int rows = chunk_rows(a.T, kNL == 32 ? kMaxBlocks : kMaxBlocks / 2);
    const int chunks = (a.T + rows - 1) / rows;
    const cudaError_t e =
        launch_pdl(router_partial_kernel<DT, kNL, kNV>, dim3(chunks), dim3(kWarps * 32),
                   (kWarps + 1) * a.E * 4, s, a, w, rows);
    if (e != cudaSuccess) return e;
    int Y = 8;  // about a thread per two slots of a sequence; 256 threads for the last block
    while (Y < 32 && 2 * Y * a.S < chunks + a.S) Y *= 2;
    // a block per sequence and 32 experts while that is not more than fill the device
    int groups = kMaxBlocks / a.S;
    groups = groups < 1 ? 1 : groups < expert_blocks(a.E) ? groups : expert_blocks(a.E);
    return launch_pdl(router_combine_kernel, dim3(a.S, groups), dim3(32, Y), 0, s, a, w, rows);
  });
}

template <int DT>
cudaError_t launch_grad(RouterLossArgs a, cudaStream_t s) {
  a.aligned = rows_aligned<DT>(a);
  a.counts_aligned = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.counts) % 16 == 0;
  return with_layout<DT>(a, [&](auto nl, auto nv) {
    constexpr int kNL = decltype(nl)::value;
    // several rows a lane once there are rows for all warps of these blocks: few blocks
    // where a lane's part of f_se is long to load
    constexpr int kBlocks = kNL == 32 ? 2 * kMaxBlocks : kMaxBlocks / 2;
    const int64_t at_once = (int64_t)kWarps * (32 / kNL);
    const int rows = (int)((a.T + at_once * kBlocks - 1) / (at_once * kBlocks));
    return launch_pdl(router_grad_kernel<DT, kNL, decltype(nv)::value>,
                      dim3((unsigned)((a.T + at_once * rows - 1) / (at_once * rows))),
                      dim3(kWarps * 32), 0, s, a, rows);
  });
}

}  // namespace

size_t router_loss_ws_bytes(int T, int E, int S) {
  return 256 + seq_bytes(S) + dots_bytes(S, E) +
         ((size_t)max_chunks(T) + S) * (2 * (size_t)E + 3) * sizeof(float);
}

cudaError_t launch_router_loss(const RouterLossArgs& a, int dtype, cudaStream_t s) {
  if (dtype == kF32) return launch_loss<kF32>(a, s);
  if (dtype == kBf16) return launch_loss<kBf16>(a, s);
  return launch_loss<kF16>(a, s);
}

cudaError_t launch_router_loss_grad(const RouterLossArgs& a, int dtype, cudaStream_t s) {
  if (dtype == kF32) return launch_grad<kF32>(a, s);
  if (dtype == kBf16) return launch_grad<kBf16>(a, s);
  return launch_grad<kF16>(a, s);
}

}  // namespace moe
