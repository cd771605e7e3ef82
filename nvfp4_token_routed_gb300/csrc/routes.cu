// routes.cu -- routes sorted by expert, token rows copied to their routes' rows and
// summed back, and the gradients of both.
//
//   sort     stable counting sort of the T*K chosen experts: offsets[e] the first row of
//            expert e, perm[r] the route of row r, inv[t][k] the row of route (t, k)
//   dispatch rows[inv[t][k]] = x[t];        its gradient is combine without weights
//   combine  out[t] = sum_k w[t][k] rows[inv[t][k]], fp32 from k = 0 on, rounded once
//   gradient drows[inv[t][k]] = w[t][k] dout[t], dw[t][k] = rows[inv[t][k]] . dout[t]
//
// All row kernels go by tokens, not by rows: a token's row is read (or written) once and
// its K rows stay independent accesses in flight, and no sum meets another thread's, so
// equal inputs give equal bits.  They are bound by HBM, the sort by latency.  Measured (bf16,
// T4096 K6 H7168, 384 experts; copy rate 6686 GB/s): dispatch 59 us (1.05 of the copy rate,
// as its last writes are still in L2), combine 66 us (0.94), its gradient 122 us (0.93), the
// sort of the 24576 routes 10 us in one launch (three launches of many blocks: 18.5), of
// 524288 and 4194304 (256 experts, three launches) 15 and 60 us; the same rows in microscaled FP4
// dispatched in 18.4 us (0.89 of the copy rate).
#include <algorithm>

#include "block32.cuh"
#include "cluster.cuh"
#include "experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- sort
// A chunk of routes is one block's: each warp takes a contiguous part, 32 routes at a
// time; votes rank equal experts within the 32, a count per warp and expert in
// shared memory carries the rank on, and a prefix over the warps makes it the chunk's.
constexpr int kChunk = 2048;      // routes a block of many
constexpr int kChunkWarps = 8;
constexpr int kOneBlock = 4096;   // routes a block of a batch that one cluster sorts
constexpr int kOneWarps = 32;
constexpr int kSmall = 1024;      // routes of the only block of a small batch
constexpr int kCluster = 8;       // blocks of the largest cluster: 32768 routes

int64_t chunks_of(int64_t TK) { return (TK + kChunk - 1) / kChunk; }

__device__ __forceinline__ int route_expert(const SortArgs& a, int i, bool& bad) {
  int e;
  if (a.ids64) {
    const int64_t v = reinterpret_cast<const int64_t*>(a.ids)[i];
    bad = v < -1 || v >= a.E;
    e = bad ? -1 : (int)v;
  } else {
    e = reinterpret_cast<const int32_t*>(a.ids)[i];
    bad = e < -1 || e >= a.E;
    if (bad) e = -1;
  }
  return e;
}

// Exclusive sum over the block's threads (blockDim.x <= 1024, a multiple of 32).
__device__ __forceinline__ int block_exclusive(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < nw; ++w) {
    const int c = s_warp[w];
    if (w < warp) before += c;
    total += c;
  }
  __syncthreads();
  return before + x - v;
}

// Ranks of a block's routes [c0, c1) and their counts.  cnt: [warps][E] in shared memory;
// on return the routes of expert e in warps before w.  Iteration j of this thread's
// route: key[j], rank[j] (within the warp's part).  total[e] of a chunk: `chunk_total`.
template <int WARPS, int ITERS>
__device__ __forceinline__ void rank_chunk(const SortArgs& a, int c0, int c1, uint16_t* cnt,
                                           int (&key)[ITERS], int (&rank)[ITERS], bool& any_bad) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* mine = cnt + warp * a.E;
  for (int e = lane; e < a.E; e += 32) mine[e] = 0;
  const int w0 = c0 + warp * (32 * ITERS);
  const int bits = 32 - __clz(a.E);  // E < 2^bits: keys 0 .. E - 1 and 2^bits - 1
  any_bad = false;
#pragma unroll
  for (int j = 0; j < ITERS; ++j) {
    const int i = w0 + 32 * j + lane;
    bool bad = false;
    key[j] = i < c1 ? route_expert(a, i, bad) : -1;
    any_bad |= bad;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < ITERS; ++j) {
    // lanes with this lane's key, a vote a bit (match.any takes a step for each of the up to
    // 32 different keys); key -1 has every bit set, and no expert has
    unsigned same = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
      const bool set = (key[j] >> b) & 1;
      const unsigned vote = __ballot_sync(0xFFFFFFFFu, set);
      same &= set ? vote : ~vote;
    }
    const int first = __ffs(same) - 1;
    int before = 0;
    if (lane == first && key[j] >= 0) {
      before = mine[key[j]];
      mine[key[j]] = (uint16_t)(before + __popc(same));
    }
    before = __shfl_sync(0xFFFFFFFFu, before, first);
    rank[j] = before + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
  }
}

__device__ __forceinline__ void write_route(const SortArgs& a, int i, int row) {
  a.inv[i] = row;
  if (row >= 0) a.perm[row] = i;
}

// The whole sort of a few routes by one block of 8 warps: no cluster, and a quarter of the
// counters (128 routes of 256 experts 4.0 us, by the cluster's kernel 8.1).
__global__ void __launch_bounds__(kChunkWarps * 32) sort_small_kernel(const SortArgs a) {
  constexpr int kIters = kSmall / (kChunkWarps * 32);
  constexpr int kPer = 1024 / (kChunkWarps * 32);  // experts a thread
  __shared__ uint16_t cnt[kChunkWarps * 1024];
  __shared__ int s_base[1024];
  __shared__ int s_warp[kChunkWarps];
  __shared__ int s_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int TK = a.T * a.K;
  if (threadIdx.x == 0) s_bad = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  int key[kIters], rank[kIters];
  bool bad;
  rank_chunk<kChunkWarps, kIters>(a, 0, TK, cnt, key, rank, bad);
  if (bad) s_bad = 1;
  __syncthreads();
  int tot[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    tot[i] = 0;
    if (e < a.E) {
      int c[kChunkWarps];
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) c[w] = cnt[w * a.E + e];
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) {
        cnt[w * a.E + e] = (uint16_t)tot[i];
        tot[i] += c[w];
      }
    }
    sum += tot[i];
  }
  int n;
  int off = block_exclusive(sum, s_warp, n);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < a.E) {
      s_base[e] = off;
      a.offsets[e] = off;
    }
    off += tot[i];
  }
  if (threadIdx.x == 0) {
    a.offsets[a.E] = n;
    if (a.status) a.status[kStatusFlags] = s_bad ? kFlagBadExpertId : 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kIters; ++j) {
    const int i = warp * (32 * kIters) + 32 * j + lane;
    if (i >= TK) continue;
    const int e = key[j];
    write_route(a, i, e < 0 ? -1 : s_base[e] + cnt[warp * a.E + e] + rank[j]);
    if (i >= n) a.perm[i] = -1;
  }
}

// Value of another block of the cluster at this block's shared address p.
__device__ __forceinline__ int load_cluster(const int* p, int rank) {
  uint32_t r;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

// The whole sort by one cluster: block c ranks routes [c kOneBlock, ...), reads the other
// blocks' counts in their shared memory, and adds up for itself where its routes go.
__global__ void __launch_bounds__(kOneWarps * 32) sort_cluster_kernel(const SortArgs a) {
  constexpr int kIters = kOneBlock / (kOneWarps * 32);
  extern __shared__ uint16_t cnt[];
  __shared__ int s_warp[kOneWarps];
  __shared__ int s_count[1025];  // this block's routes of each expert; [E]: a bad id
  __shared__ int s_base[1024];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_rank(), blocks = (int)cluster_size();
  const int TK = a.T * a.K, c0 = rank * kOneBlock;
  if (threadIdx.x == 0) s_count[a.E] = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  int key[kIters], row[kIters];
  bool bad;
  rank_chunk<kOneWarps, kIters>(a, c0, min(TK, c0 + kOneBlock), cnt, key, row, bad);
  if (bad) s_count[a.E] = 1;
  __syncthreads();
  // thread e: expert e's routes in each warp's part
  const int e = threadIdx.x;
  if (e < a.E) {
    int c[kOneWarps], sum = 0;  // all reads before the writes: they overlap
#pragma unroll
    for (int w = 0; w < kOneWarps; ++w) c[w] = cnt[w * a.E + e];
#pragma unroll
    for (int w = 0; w < kOneWarps; ++w) {
      cnt[w * a.E + e] = (uint16_t)sum;
      sum += c[w];
    }
    s_count[e] = sum;
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  int before = 0, total = 0;
  if (e < a.E) {
    int v[kCluster];
#pragma unroll
    for (int c = 0; c < kCluster; ++c) v[c] = c < blocks ? load_cluster(s_count + e, c) : 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
      if (c < rank) before += v[c];
      total += v[c];
    }
  }
  int any_bad = 0;
  if (rank == 0 && threadIdx.x == 0)
    for (int c = 0; c < blocks; ++c) any_bad |= load_cluster(s_count + a.E, c);
  __syncwarp();
  cluster_arrive();  // no more reads of other blocks
  int n;
  const int off = block_exclusive(total, s_warp, n);
  if (e < a.E) {
    s_base[e] = off + before;
    if (rank == 0) a.offsets[e] = off;
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.offsets[a.E] = n;
    if (a.status) a.status[kStatusFlags] = any_bad ? kFlagBadExpertId : 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kIters; ++j) {
    const int i = c0 + warp * (32 * kIters) + 32 * j + lane;
    if (i >= TK) continue;
    const int k = key[j];
    write_route(a, i, k < 0 ? -1 : s_base[k] + cnt[warp * a.E + k] + row[j]);
    if (i >= n) a.perm[i] = -1;
  }
  __syncwarp();
  cluster_wait();
}

// Counts of each chunk, and whether it held a bad id.
__global__ void __launch_bounds__(kChunkWarps * 32) sort_count_kernel(const SortArgs a) {
  __shared__ int cnt[1025];
  const int TK = a.T * a.K;
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) cnt[e] = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  const int c0 = blockIdx.x * kChunk, c1 = min(TK, c0 + kChunk);
  for (int i = c0 + threadIdx.x; i < c1; i += blockDim.x) {
    bool bad = false;
    const int e = route_expert(a, i, bad);
    if (e >= 0) atomicAdd(&cnt[e], 1);
    if (bad) cnt[a.E] = 1;
  }
  __syncthreads();
  int32_t* dst = a.chunks + (int64_t)blockIdx.x * (a.E + 1);
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) dst[e] = cnt[e];
}

// Each column of chunk counts replaced by its exclusive sums; totals behind the chunks.
// Lane = column, so that a warp reads 128 bytes of a chunk; 32 warps share the chunks.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const SortArgs a, int n_chunks) {
  __shared__ int part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, stride = a.E + 1;
  const int per = (n_chunks + 31) / 32;
  const int k0 = min(n_chunks, warp * per), k1 = min(n_chunks, k0 + per);
  pdl_trigger();
  pdl_wait();
  int sum = 0;
  if (col <= a.E)
    for (int k = k0; k < k1; ++k) sum += a.chunks[(int64_t)k * stride + col];
  part[warp][lane] = sum;
  __syncthreads();
  int run = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const int c = part[w][lane];
    if (w < warp) run += c;
    total += c;
  }
  if (col > a.E) return;
  if (col < a.E)
    for (int k = k0; k < k1; ++k) {
      int32_t* p = a.chunks + (int64_t)k * stride + col;
      const int c = *p;
      *p = run;
      run += c;
    }
  if (warp != 0) return;
  if (col < a.E)
    a.chunks[(int64_t)n_chunks * stride + col] = total;
  else
    a.status[kStatusFlags] = total ? kFlagBadExpertId : 0;
}

// Rows of each chunk's routes.  Every block adds the experts' totals up for itself.
__global__ void __launch_bounds__(kChunkWarps * 32) sort_place_kernel(const SortArgs a,
                                                                      int n_chunks) {
  constexpr int kIters = kChunk / (kChunkWarps * 32);
  constexpr int kPer = 1024 / (kChunkWarps * 32);  // experts a thread
  __shared__ uint16_t cnt[kChunkWarps * 1024];
  __shared__ int s_base[1024];
  __shared__ int s_warp[kChunkWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int TK = a.T * a.K, stride = a.E + 1;
  const int c0 = blockIdx.x * kChunk, c1 = min(TK, c0 + kChunk);
  pdl_trigger();
  pdl_wait();
  int key[kIters], rank[kIters];
  bool bad;
  rank_chunk<kChunkWarps, kIters>(a, c0, c1, cnt, key, rank, bad);
  const int32_t* totals = a.chunks + (int64_t)n_chunks * stride;
  int tot[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    tot[i] = e < a.E ? totals[e] : 0;
    sum += tot[i];
  }
  int n;
  int off = block_exclusive(sum, s_warp, n);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < a.E) {
      s_base[e] = off + a.chunks[(int64_t)blockIdx.x * stride + e];
      if (blockIdx.x == 0) a.offsets[e] = off;
      int run = 0;
      for (int w = 0; w < kChunkWarps; ++w) {
        const int c = cnt[w * a.E + e];
        cnt[w * a.E + e] = (uint16_t)run;
        run += c;
      }
    }
    off += tot[i];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = n;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kIters; ++j) {
    const int i = c0 + warp * (32 * kIters) + 32 * j + lane;
    if (i >= c1) continue;
    const int e = key[j];
    write_route(a, i, e < 0 ? -1 : s_base[e] + cnt[warp * a.E + e] + rank[j]);
    if (i >= n) a.perm[i] = -1;
  }
}

// ---------------------------------------------------------------- rows
template <int VB>
struct VecOf;
template <>
struct VecOf<16> {
  using type = uint4;
};
template <>
struct VecOf<8> {
  using type = uint2;
};
template <>
struct VecOf<4> {
  using type = uint32_t;
};
template <>
struct VecOf<2> {
  using type = uint16_t;
};

// The row of route (t, k); -1 for an empty slot and for anything that is no row.
__device__ __forceinline__ int route_row(const RowArgs& a, int64_t i) {
  const int r = a.inv[i];
  return (unsigned)r < (unsigned)(a.T * a.K) ? r : -1;
}

// Token and vector of a flat index; 64-bit division only where the index needs it.
__device__ __forceinline__ int split_index(int64_t i, int vecs, int& v) {
  const int t = i <= 0xFFFFFFFFll ? (int)((uint32_t)i / (uint32_t)vecs) : (int)(i / vecs);
  v = (int)(i - (int64_t)t * vecs);
  return t;
}

// One thread a vector of a token's row: read once, written K times.
template <int VB>
__global__ void __launch_bounds__(256) dispatch_kernel(const RowArgs a, int64_t ld_in,
                                                       int64_t ld_out, int vecs) {
  using V = typename VecOf<VB>::type;
  pdl_trigger();
  int v;
  const int t = split_index((int64_t)blockIdx.x * 256 + threadIdx.x, vecs, v);
  if (t >= a.T) return;
  pdl_wait();
  const V x = reinterpret_cast<const V*>(a.x)[t * ld_in + v];
  V* out = reinterpret_cast<V*>(a.out) + v;
  for (int k = 0; k < a.K; ++k) {
    const int r = route_row(a, (int64_t)t * a.K + k);
    if (r >= 0) out[r * ld_out] = x;
  }
}

// A microscaled matrix: a row's codes as vectors of 16 bytes, then its 8 bytes of each scale
// panel, one thread each.
__global__ void __launch_bounds__(256) dispatch_mx_kernel(const RowArgs a, int code_vecs,
                                                          int panels, const uint2* scales,
                                                          uint2* out_scales) {
  pdl_trigger();
  int v;
  const int t = split_index((int64_t)blockIdx.x * 256 + threadIdx.x, code_vecs + panels, v);
  if (t >= a.T) return;
  pdl_wait();
  if (v < code_vecs) {
    const uint4 x = reinterpret_cast<const uint4*>(a.x)[(int64_t)t * code_vecs + v];
    uint4* out = reinterpret_cast<uint4*>(a.out) + v;
    for (int k = 0; k < a.K; ++k) {
      const int r = route_row(a, (int64_t)t * a.K + k);
      if (r >= 0) out[(int64_t)r * code_vecs] = x;
    }
    return;
  }
  const int64_t p = v - code_vecs;
  const int64_t in_rows = (a.T + 1) & ~1, out_rows = ((int64_t)a.T * a.K + 1) & ~int64_t(1);
  const uint2 x = scales[p * in_rows + t];
  for (int k = 0; k < a.K; ++k) {
    const int r = route_row(a, (int64_t)t * a.K + k);
    if (r >= 0) out_scales[p * out_rows + r] = x;
  }
}

template <int DT, int VB>
struct RowVec {
  static constexpr int kSize = DT == kF32 ? 4 : 2;
  static constexpr int kN = VB / kSize;
  using V = typename VecOf<VB>::type;
  __device__ static __forceinline__ void unpack(const V& v, float (&f)[kN]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
    if constexpr (VB == 2) {
      f[0] = elem_to_float<DT>(*reinterpret_cast<const uint16_t*>(&v));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        f[i] = DT == kF32 ? __uint_as_float(w[i])
                          : elem_to_float<DT>((w[i * kSize / 4] >> (16 * (i & 1))) & 0xFFFFu);
    }
  }
  __device__ static __forceinline__ V pack(const float (&f)[kN]) {
    V v;
    if constexpr (VB == 2) {
      v = (uint16_t)float_to_elem<DT>(f[0]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < VB / 4; ++i)
        w[i] = DT == kF32 ? float_to_elem<DT>(f[i % kN])
                          : float_to_elem<DT>(f[(2 * i) % kN]) |
                                (float_to_elem<DT>(f[(2 * i + 1) % kN]) << 16);
    }
    return v;
  }
};

// TPT threads a token, each a vector of its output at a time.  ROWS routes at a time: their
// row numbers and weights (once a token where K <= ROWS), then their vectors, all in flight,
// then the sum.  ROWS = K has kernels of its own where rows lie on 16 bytes.
template <int DT, int VB, int ROWS, int TPT>
__global__ void __launch_bounds__(256) combine_kernel(const RowArgs a, int64_t ld_in,
                                                      int64_t ld_out, int vecs) {
  using RV = RowVec<DT, VB>;
  using V = typename RV::V;
  const int t = blockIdx.x * (256 / TPT) + threadIdx.x / TPT;
  pdl_trigger();
  if (t >= a.T) return;
  pdl_wait();
  int r[ROWS];
  float w[ROWS];
  auto routes = [&](int k0) {
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t route = (int64_t)t * a.K + k0 + u;
      r[u] = k0 + u < a.K ? route_row(a, route) : -1;
      w[u] = 1.0f;
      if (a.w && r[u] >= 0) w[u] = a.w[route];
    }
  };
  routes(0);
  for (int v = threadIdx.x % TPT; v < vecs; v += TPT) {
    const V* in = reinterpret_cast<const V*>(a.x) + v;
    float acc[RV::kN];
#pragma unroll
    for (int j = 0; j < RV::kN; ++j) acc[j] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += ROWS) {
      if (a.K > ROWS) routes(k0);
      V y[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u)
        if (r[u] >= 0) y[u] = in[r[u] * ld_in];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        float f[RV::kN];
        RV::unpack(y[u], f);
        if (r[u] >= 0) {
#pragma unroll
          for (int j = 0; j < RV::kN; ++j) acc[j] = fmaf(w[u], f[j], acc[j]);
        }
      }
    }
    reinterpret_cast<V*>(a.out)[t * ld_out + v] = RV::pack(acc);
  }
}

// Gradient of combine.  A block holds kTokens tokens of TPT threads each.  A thread keeps
// up to kVecs vectors of dout in registers and walks the K routes: row read, its product
// summed over the warp, w dout written.
constexpr int kGradVecs = 4;
template <int DT, int VB, int TPT>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowArgs a, int64_t ld_in,
                                                           int64_t ld_dout, int64_t ld_out,
                                                           int vecs) {
  using RV = RowVec<DT, VB>;
  using V = typename RV::V;
  constexpr int kTokens = 256 / TPT, kWarps = TPT / 32;
  __shared__ float s_dot[kTokens][kWarps][32];  // [k]
  const int sub = threadIdx.x / TPT, tid = threadIdx.x % TPT;
  const int lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x * kTokens + sub;
  pdl_trigger();
  s_dot[sub][warp][lane] = 0.0f;
  __syncwarp();
  pdl_wait();
  if (t < a.T) {
    for (int v0 = tid; v0 - tid < vecs; v0 += TPT * kGradVecs) {
      float d[kGradVecs][RV::kN];
#pragma unroll
      for (int u = 0; u < kGradVecs; ++u) {
        const int v = v0 + u * TPT;
        if (v < vecs)
          RV::unpack(reinterpret_cast<const V*>(a.dout)[t * ld_dout + v], d[u]);
        else
#pragma unroll
          for (int j = 0; j < RV::kN; ++j) d[u][j] = 0.0f;
      }
      for (int k = 0; k < a.K; ++k) {
        const int64_t route = (int64_t)t * a.K + k;
        const int r = route_row(a, route);  // the same for every thread of the token
        if (r < 0) continue;
        const float w = a.w ? a.w[route] : 1.0f;
        float dot = 0.0f;
        if (a.x) {
          V y[kGradVecs];
#pragma unroll
          for (int u = 0; u < kGradVecs; ++u)
            if (v0 + u * TPT < vecs)
              y[u] = reinterpret_cast<const V*>(a.x)[r * ld_in + v0 + u * TPT];
#pragma unroll
          for (int u = 0; u < kGradVecs; ++u)
            if (v0 + u * TPT < vecs) {
              float f[RV::kN];
              RV::unpack(y[u], f);
#pragma unroll
              for (int j = 0; j < RV::kN; ++j) dot = fmaf(f[j], d[u][j], dot);
            }
        }
#pragma unroll
        for (int u = 0; u < kGradVecs; ++u)
          if (v0 + u * TPT < vecs) {
            float g[RV::kN];
#pragma unroll
            for (int j = 0; j < RV::kN; ++j) g[j] = w * d[u][j];
            reinterpret_cast<V*>(a.out)[r * ld_out + v0 + u * TPT] = RV::pack(g);
          }
        if (a.x) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
          if (lane == 0) s_dot[sub][warp][k] += dot;
        }
      }
    }
  }
  if (!a.dw) return;
  __syncthreads();
  if (t < a.T && tid < a.K) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_dot[sub][w][tid];
    a.dw[(int64_t)t * a.K + tid] = sum;
  }
}

int64_t blocks_of(int64_t threads) { return (threads + 255) / 256; }
int dtype_size(int dtype) { return dtype == kF32 ? 4 : 2; }

}  // namespace

size_t sort_routes_ws_bytes(int64_t TK, int E) {
  if (TK <= kCluster * kOneBlock) return kSortStatusBytes;
  return kSortStatusBytes + sizeof(int32_t) * ((size_t)chunks_of(TK) * (E + 1) + E);
}

cudaError_t launch_sort_routes(const SortArgs& a, cudaStream_t s) {
  const int64_t TK = (int64_t)a.T * a.K;
  if (TK <= kSmall)
    return launch_pdl(sort_small_kernel, dim3(1), dim3(kChunkWarps * 32), 0, s, a);
  if (TK <= kCluster * kOneBlock) {
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(sort_cluster_kernel),
                                      kOneWarps * 1024 * 2, configured);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((TK + kOneBlock - 1) / kOneBlock);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kOneWarps * 32);
    cfg.dynamicSmemBytes = (size_t)kOneWarps * a.E * 2;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sort_cluster_kernel, a);
  }
  const int n = (int)chunks_of(TK);
  cudaError_t e = launch_pdl(sort_count_kernel, dim3(n), dim3(kChunkWarps * 32), 0, s, a);
  if (e == cudaSuccess)
    e = launch_pdl(sort_scan_kernel, dim3((a.E + 1 + 31) / 32), dim3(1024), 0, s, a, n);
  if (e == cudaSuccess)
    e = launch_pdl(sort_place_kernel, dim3(n), dim3(kChunkWarps * 32), 0, s, a, n);
  return e;
}

cudaError_t launch_dispatch(const RowArgs& a, int dtype, cudaStream_t s) {
  const int sz = dtype_size(dtype);
  const int64_t row = (int64_t)a.H * sz;
  const int vb = std::min(access_bytes(a.x, a.ld_x * sz, row),
                          access_bytes(a.out, a.ld_out * sz, row));
  const int vecs = (int)(row / vb);
  const dim3 grid((unsigned)blocks_of((int64_t)a.T * vecs));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, s, a, a.ld_x * sz / vb, a.ld_out * sz / vb, vecs);
  };
  switch (vb) {
    case 16: return go(dispatch_kernel<16>);
    case 8: return go(dispatch_kernel<8>);
    case 4: return go(dispatch_kernel<4>);
    default: return go(dispatch_kernel<2>);
  }
}

cudaError_t launch_dispatch_mx(const RowArgs& a, const uint8_t* scales, uint8_t* out_scales,
                               cudaStream_t s) {
  const int code_vecs = a.H / 32, panels = a.H / kMxPanel;
  const dim3 grid((unsigned)blocks_of((int64_t)a.T * (code_vecs + panels)));
  return launch_pdl(dispatch_mx_kernel, grid, dim3(256), 0, s, a, code_vecs, panels,
                    reinterpret_cast<const uint2*>(scales), reinterpret_cast<uint2*>(out_scales));
}

namespace {

template <int DT, int VB, int ROWS>
cudaError_t combine_rows(const RowArgs& a, cudaStream_t s) {
  const int sz = dtype_size(DT);
  const int vecs = (int)((int64_t)a.H * sz / VB);
  auto go = [&](auto kernel, int tpt) {
    const int tokens = 256 / tpt;
    return launch_pdl(kernel, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(256), 0, s, a,
                      a.ld_x * sz / VB, a.ld_out * sz / VB, vecs);
  };
  // a block a token where its row fills one, or where tokens are too few to fill the device
  if (vecs > 128 || (vecs > 32 && a.T < 152 * 8)) return go(combine_kernel<DT, VB, ROWS, 256>, 256);
  return go(combine_kernel<DT, VB, ROWS, 32>, 32);
}

template <int DT>
cudaError_t combine_typed(const RowArgs& a, cudaStream_t s) {
  const int sz = dtype_size(DT);
  const int64_t row = (int64_t)a.H * sz;
  const int vb = std::min(access_bytes(a.x, a.ld_x * sz, row),
                          access_bytes(a.out, a.ld_out * sz, row));
  if (vb == 16) {
    switch (a.K) {
      case 1: return combine_rows<DT, 16, 1>(a, s);
      case 2: return combine_rows<DT, 16, 2>(a, s);
      case 6: return combine_rows<DT, 16, 6>(a, s);
      case 8: return combine_rows<DT, 16, 8>(a, s);
      default: return combine_rows<DT, 16, 4>(a, s);
    }
  }
  if (vb == 8) return combine_rows<DT, 8, 4>(a, s);
  if (vb == 4) return combine_rows<DT, 4, 4>(a, s);
  if constexpr (DT != kF32) return combine_rows<DT, 2, 4>(a, s);
  return cudaErrorInvalidValue;
}

template <int DT, int VB>
cudaError_t combine_grad_vb(const RowArgs& a, cudaStream_t s) {
  const int sz = dtype_size(DT);
  const int vecs = (int)((int64_t)a.H * sz / VB);
  auto go = [&](auto kernel, int tpt) {
    const int tokens = 256 / tpt;
    return launch_pdl(kernel, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(256), 0, s, a,
                      a.ld_x * sz / VB, a.ld_dout * sz / VB, a.ld_out * sz / VB, vecs);
  };
  // as many threads a token as its row has vectors for
  if (vecs <= 32 * kGradVecs) return go(combine_grad_kernel<DT, VB, 32>, 32);
  if (vecs <= 64 * kGradVecs) return go(combine_grad_kernel<DT, VB, 64>, 64);
  if (vecs <= 128 * kGradVecs) return go(combine_grad_kernel<DT, VB, 128>, 128);
  return go(combine_grad_kernel<DT, VB, 256>, 256);
}

template <int DT>
cudaError_t combine_grad_typed(const RowArgs& a, cudaStream_t s) {
  const int sz = dtype_size(DT);
  const int64_t row = (int64_t)a.H * sz;
  int vb = std::min(access_bytes(a.dout, a.ld_dout * sz, row),
                    access_bytes(a.out, a.ld_out * sz, row));
  if (a.x) vb = std::min(vb, access_bytes(a.x, a.ld_x * sz, row));
  switch (vb) {
    case 16: return combine_grad_vb<DT, 16>(a, s);
    case 8: return combine_grad_vb<DT, 8>(a, s);
    case 4: return combine_grad_vb<DT, 4>(a, s);
    default: break;
  }
  if constexpr (DT != kF32) return combine_grad_vb<DT, 2>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_combine(const RowArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? combine_typed<kF32>(a, s)
         : dtype == kBf16 ? combine_typed<kBf16>(a, s)
                          : combine_typed<kF16>(a, s);
}
cudaError_t launch_combine_grad(const RowArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? combine_grad_typed<kF32>(a, s)
         : dtype == kBf16 ? combine_grad_typed<kBf16>(a, s)
                          : combine_grad_typed<kF16>(a, s);
}

}  // namespace moe
