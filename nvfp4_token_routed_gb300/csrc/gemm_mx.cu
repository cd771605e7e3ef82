// gemm_mx.cu -- product of microscaled FP4 rows with their expert's weights:
//   y[r][n] = sum_d x[r][d] w[e(r)][n][d],  both E2M1 with a power of two per 32 values,
// on tcgen05 tensor cores (kind::mxf4, K = 64 an instruction, fp32 accumulators in TMEM).
// Rows lie sorted by expert (or form one group); groups start at any row.
//
// Weights are the M = 128 operand and rows the N operand, so that the few rows of a
// decode step do not leave a 128-row instruction idle.  Bounds: a launch reads each
// used weight once (17/32 byte a value) and is bound by HBM up to some 500 rows an
// expert, beyond by what the tensor cores are fed with.
//
//   * Persistent CTAs, one an SM.  Work item = (tile of up to 192 rows of one expert,
//     128-row weight tile); a group's rows are cut into equal tiles of whole 16s.  Items
//     are numbered expert by expert and weight-tile-major, so that the row tiles of one
//     weight tile run next to each other and it comes from HBM once.  Every CTA adds the
//     groups up for itself and takes items blockIdx.x, + gridDim.x, ...: no counter, no
//     workspace, nothing to reset between launches.
//   * Warp 0 loads weight tiles (TMA, 128-byte swizzle) and their scales, warp 10 row
//     tiles (a box, two above 128 rows: a map for each height) and theirs; a stage is 256
//     values deep.  A stage's scales are one contiguous piece of a panel (mx_quant.cu), which
//     starts on an even row: 8 bytes a row, 16 a bulk copy's boundary.
//   * Warps 6-9 move a stage's scales to TMEM: row r at lane r % 32, column r / 32, in
//     all four lane quadrants; one 32-bit column holds 128 values' four scales, and the
//     instruction takes two of them by its scale id.
//   * Warp 1 issues the MMAs, warps 2-5 drain the accumulators (two, or four where no
//     tile passes 64 rows): a lane holds one output feature, four lanes exchange so that
//     every store is 8 bytes of one row.
//   * Waits are bounded.  A CTA in which one runs out drains its copies and MMAs, frees
//     TMEM, and writes NaN to the items that it leaves.
// Measured (bf16 out): 128 rows on 64 experts N2048 D2048 22.2 us (0.97 of the copy rate,
// 6686 GB/s), on 256 experts N4096 D7168 223 us (1.0); 2048 rows on 32 experts N4096 D7168 83
// us (0.95).  One matrix N4096 D7168 has 32 items and is bound by how fast 32 CTAs read: 1 to 16
// rows 9.3 us (floor 2.4).  Where rows bound it, see the pairs below.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include <cstdint>

#include "block32.cuh"
#include "cluster.cuh"
#include "experts.h"
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kRowBytes = kMxPanel / 2;        // code bytes of a row and stage
constexpr int kABytes = 128 * kRowBytes;
constexpr int kSfaBytes = 1152;                // 130 rows of 8 bytes, padded
constexpr int kTileN = 192;                    // rows of the largest tile
constexpr int kStages = 12;                    // at most
constexpr int kAccs = 4;
constexpr int kTmemCols = 512;
constexpr int kSmem = 227 * 1024;
constexpr int kThreads = 352;                  // 11 warps
// mbarriers
constexpr int kFull = 0;
constexpr int kEmpty = kStages;
constexpr int kSfReady = 2 * kStages;
constexpr int kAccFull = 3 * kStages;
constexpr int kAccEmpty = kAccFull + kAccs;
constexpr int kDrain = kAccEmpty + kAccs;
constexpr int kBars = kDrain + 1;
constexpr int kFlagsOff = 8 * kBars;           // tmem slot, abort flag, -, tile height
constexpr int kWarpSumOff = kFlagsOff + 32;    // an int a warp
constexpr int kGroupsOff = 512;                // first item [E + 1], first row [E + 1]
static_assert(kWarpSumOff + 4 * (kThreads / 32) <= kGroupsOff, "barrier area");

// CTAs work in pairs from this many rows an expert and stages a row on (both measured, us,
// single / pair): N4096 D7168, 8 experts of 192 rows 27.9 / 32.2, of 256 39.5 / 33.2, of 1024
// 108 / 76; N7168 D2048, 32 experts of 256 77 / 64, of 1024 239 / 191; N2048 D1024, 8 experts
// of 256 9.2 / 9.9, of 1024 19.4 / 19.6.  Few items leave pairs idle: one matrix N4096 D7168,
// 256 rows 11.5 / 15.0 (16 items of pairs), 512 15.1 / 15.4, 1024 24.3 / 16.5.  One weight
// tile leaves half of a pair idle: R16384 D2048 N128 9.0 / 10.6, N256 12.0 / 10.5.
constexpr int64_t kPairRows = 224;
constexpr int kPairStages = 8;

struct MxMaps {
  CUtensorMap w;
  CUtensorMap x[8];  // 16, 32, ... 128 rows
};

// A value that is the same in every lane, and that the compiler then knows to be: what
// depends on it (branches, descriptors, addresses of copies) stays in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Two values as 16-bit elements, a in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint2 lds64(uint32_t saddr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(saddr));
  return v;
}

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, UE8M0 scales, K-major operands.
__device__ __forceinline__ uint32_t idesc_mxf4(uint32_t M, uint32_t N) {
  return (1u << 7) | (1u << 10) | (((N >> 3) & 0x3F) << 17) | (1u << 23) |
         (((M >> 4) & 0x1F) << 24);
}
// By a converged warp; the elected lane issues.
__device__ __forceinline__ void mma_mxf4_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// Issue of a stage's copies by a converged warp with warp-uniform operands: the elected
// lane announces the stage's bytes (expect) and copies a box of codes and a piece of scales.
// In a branch of one lane each copy costs its thread a few hundred cycles.
__device__ __forceinline__ void expect_warp(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void box_warp(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                         int32_t c0, int32_t c1, uint64_t policy) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void piece_warp(uint32_t dst, const void* src, uint32_t bytes,
                                           uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2,"
      " [%3];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool wait_or_leave(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// After an abort: wait (one shared time limit) for the last phases of the ring that this
// warp has loaded, so that no copy lands in shared memory once the CTA is gone.  A phase
// that the other producer never joined does not complete; the limit ends the wait, by which
// time this warp's copies have landed.
__device__ __forceinline__ void drain_ring(const Ring& R, int loaded, int n_stages) {
  const uint64_t t0 = globaltimer();
  for (int i = max(0, loaded - n_stages); i < loaded; ++i)
    while (!mbar_try_wait_sleep(R.bar(kFull + i % n_stages), (uint32_t)(i / n_stages) & 1u))
      if (globaltimer() - t0 > kWaitLimitNs) return;
}

// At the end of a walk, by the warp that loads weights: the last use of each stage has been given
// back, so that no arrival of a commit is on its way to this CTA's barriers when it leaves (the
// commit behind them, on the accumulator's barrier, promises that of the MMAs alone).
__device__ __forceinline__ void await_ring(const Ring& R, int empty, int loaded, int n_stages,
                                           volatile int* abort_flag) {
  for (int i = max(0, loaded - n_stages); i < loaded; ++i)
    if (!wait_or_leave(R.bar(empty + i % n_stages), (uint32_t)(i / n_stages) & 1u, abort_flag))
      return;
}

// A CTA's walk over its items, by a whole warp.
struct Item {
  int e, mt;
  int row0, rows;  // first row of the tile, rows
};
struct Walk {
  const int* first_item;  // [E + 1]
  const int* first_row;   // [E + 1], the last one past the last group
  int m_tiles, unit, e;
  // Row tiles of a group are equal and whole units.
  __device__ __forceinline__ Item at(int item) {
    while (item >= uniform(first_item[e + 1])) ++e;
    const int i0 = uniform(first_item[e]), r0 = uniform(first_row[e]);
    const int tiles = (uniform(first_item[e + 1]) - i0) / m_tiles;
    const int group = uniform(first_row[e + 1]) - r0;
    const int h = ((group + tiles - 1) / tiles + unit - 1) & -unit;
    const int mt = (item - i0) / tiles, tt = item - i0 - mt * tiles;
    return Item{e, mt, r0 + tt * h, min(h, group - tt * h)};
  }
};

// First row of expert e; rows outside [0, R] are no rows.
__device__ __forceinline__ int group_bound(const MxGemmArgs& a, int e) {
  return a.offsets ? max(0, min(a.R, a.offsets[e])) : e ? a.R : 0;
}

// First item and first row of each expert, by the whole block (blockDim.x = THREADS): row
// tiles of at most tile_n rows in whole units of `unit`, m_tiles weight tiles each.  Also
// folds the largest tile height into *s_most (set before).  s_sum: an int a warp.
template <int THREADS>
__device__ __forceinline__ void lay_out_groups(const MxGemmArgs& a, int tile_n, int unit,
                                               int m_tiles, int* first_item, int* first_row,
                                               int* s_sum, int* s_most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.E + THREADS - 1) / THREADS;
  const int e0 = min(a.E, (int)threadIdx.x * per), e1 = min(a.E, e0 + per);
  int items = 0, most = unit;
  for (int e = e0; e < e1; ++e) {
    const int rows = max(0, group_bound(a, e + 1) - group_bound(a, e));
    const int tiles = (rows + tile_n - 1) / tile_n;
    items += tiles * m_tiles;
    if (tiles) most = max(most, ((rows + tiles - 1) / tiles + unit - 1) / unit * unit);
  }
  int x = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  atomicMax(s_most, most);
  __syncthreads();
  int before = x - items;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  for (int e = e0; e < e1; ++e) {
    const int b0 = group_bound(a, e), rows = max(0, group_bound(a, e + 1) - b0);
    first_item[e] = before;
    first_row[e] = b0;
    before += (rows + tile_n - 1) / tile_n * m_tiles;
    if (e == a.E - 1) {
      first_item[a.E] = before;
      first_row[a.E] = b0 + rows;
    }
  }
  __syncthreads();
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ MxMaps maps, const __grid_constant__ MxGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const Ring R{smem};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kFlagsOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_max16 = reinterpret_cast<int*>(tmem_slot + 3);
  int* s_sum = reinterpret_cast<int*>(smem + kWarpSumOff);
  int* first_item = reinterpret_cast<int*>(smem + kGroupsOff);
  int* first_row = first_item + a.E + 1;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int m_tiles = (a.N + 127) / 128;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(R.bar(kFull + s), 2);  // both producers
      mbar_init(R.bar(kEmpty + s), 1);
      mbar_init(R.bar(kSfReady + s), 4);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(R.bar(kAccFull + b), 1);
      mbar_init(R.bar(kAccEmpty + b), 128);
    }
    mbar_init(R.bar(kDrain), 1);
    *abort_flag = 0;
    *s_max16 = 16;
    fence_barrier_init();
    prefetch_tmap(&maps.w);
    for (int i = 0; i < 8; ++i) prefetch_tmap(&maps.x[i]);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_wait();
  pdl_trigger();

  lay_out_groups<kThreads>(a, kTileN, 16, m_tiles, first_item, first_row, s_sum, s_max16);
  const int n_items = uniform(first_item[a.E]);

  // ---- geometry from the largest tile
  const int max16 = uniform(*s_max16);
  const int acc_stride = (max16 + 31) & ~31;
  const int sfb_bytes = (8 * (acc_stride + 2) + 127) & ~127;  // read in whole 32s, from an odd row on
  const int off_b = kABytes, off_sfa = off_b + max16 * kRowBytes, off_sfb = off_sfa + kSfaBytes;
  const int stage_bytes = (off_sfb + sfb_bytes + 1023) & ~1023;
  const int nbuf = max16 <= 64 ? 4 : 2;
  const int nrb = max16 <= 128 ? 4 : 8;       // 32-row columns of a row tile's scales
  const int slot_cols = 8 + 2 * nrb;
  const int sf_base = nbuf * acc_stride;
  const int head = (kGroupsOff + 8 * (a.E + 1) + 1023) & ~1023;
  uint8_t* stages = smem + head;
  int n_stages = min(kStages, (kSmem - 1024 - head) / stage_bytes);
  n_stages = min(n_stages, (kTmemCols - sf_base) / slot_cols);

  Walk walk{first_item, first_row, m_tiles, 16, 0};
  if (warp == 0) {
    // ------------------------------------------------------------ weight producer
    const uint64_t once = policy_evict_first(), keep = policy_evict_last();
    const int64_t w_rows = ((int64_t)a.E * a.N + 1) & ~int64_t(1);
    int stage = 0, loaded = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
      const Item it = walk.at(item);
      // a weight tile of one row tile is not read again
      const uint64_t pol = first_item[it.e + 1] - first_item[it.e] == m_tiles ? once : keep;
      const int64_t row = (int64_t)it.e * a.N + it.mt * 128, r0 = row & ~int64_t(1);
      const uint32_t sf = 8u * (uint32_t)min((int64_t)(row != r0 ? 130 : 128), w_rows - r0);
      for (int kb = 0; kb < a.kblocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(kEmpty + stage), phase ^ 1, abort_flag));
        if (!ok) break;
        const uint32_t sb = smem_u32(stages + stage * stage_bytes), full = R.bar(kFull + stage);
        expect_warp(full, kABytes + sf);
        box_warp(sb, &maps.w, full, kb * kRowBytes, (int)row, pol);
        piece_warp(sb + off_sfa, a.sw + kb * a.sw_panel + 8 * r0, sf, full);
        ++loaded;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (ok) await_ring(R, kEmpty, loaded, n_stages, abort_flag);
    if (!ok || *abort_flag) drain_ring(R, loaded, n_stages);
  } else if (warp == 10) {
    // ------------------------------------------------------------ row producer
    const uint64_t pol = policy_evict_last();
    const int rows_p = (a.R + 1) & ~1;
    int stage = 0, loaded = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
      if (item == a.leave_item) break;
      const Item it = walk.at(item);
      const int n16 = (it.rows + 15) & ~15, r0 = it.row0 & ~1;
      const uint32_t sf = 8u * (uint32_t)min(n16 + (it.row0 != r0 ? 2 : 0), rows_p - r0);
      for (int kb = 0; kb < a.kblocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(kEmpty + stage), phase ^ 1, abort_flag));
        if (!ok) break;
        const uint32_t sb = smem_u32(stages + stage * stage_bytes), full = R.bar(kFull + stage);
        expect_warp(full, n16 * kRowBytes + sf);
        const int first = min(n16, 128);
        box_warp(sb + off_b, &maps.x[first / 16 - 1], full, kb * kRowBytes, it.row0, pol);
        if (n16 > 128)
          box_warp(sb + off_b + 128 * kRowBytes, &maps.x[(n16 - 128) / 16 - 1], full,
                   kb * kRowBytes, it.row0 + 128, pol);
        piece_warp(sb + off_sfb, a.sx + kb * a.sx_panel + 8 * (int64_t)r0, sf, full);
        ++loaded;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok || *abort_flag) drain_ring(R, loaded, n_stages);
  } else if (warp >= 6) {
    // ------------------------------------------------------------ scales to TMEM
    const uint32_t lane_q = (uint32_t)((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
      const Item it = walk.at(item);
      const int odd_w = (int)(((int64_t)it.e * a.N) & 1), odd_x = it.row0 & 1;
      for (int kb = 0; kb < a.kblocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(kFull + stage), phase, abort_flag));
        if (!ok) break;
        tc_fence_after();  // behind the MMAs that read this stage's columns (kEmpty, then kFull)
        const uint32_t sb = smem_u32(stages + stage * stage_bytes);
        const uint32_t col = tmem + lane_q + sf_base + stage * slot_cols;
        const uint32_t sa = sb + off_sfa + 8 * (odd_w + lane), sx = sb + off_sfb + 8 * (odd_x + lane);
        {
          const uint2 p0 = lds64(sa), p1 = lds64(sa + 256), p2 = lds64(sa + 512),
                      p3 = lds64(sa + 768);
          tmem_st4(col, make_uint4(p0.x, p1.x, p2.x, p3.x));
          tmem_st4(col + 4, make_uint4(p0.y, p1.y, p2.y, p3.y));
        }
        for (int b = 0; b < nrb; b += 4) {
          if (32 * b >= it.rows) break;
          // rows past the tile's are read from what lies there: only their own, unstored
          // columns would see them
          uint2 p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            p[j] = 32 * (b + j) < it.rows ? lds64(sx + 256 * (b + j)) : make_uint2(0u, 0u);
          tmem_st4(col + 8 + b, make_uint4(p[0].x, p[1].x, p[2].x, p[3].x));
          tmem_st4(col + 8 + nrb + b, make_uint4(p[0].y, p[1].y, p[2].y, p[3].y));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(R.bar(kSfReady + stage));
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0, local = 0;
    uint32_t phase = 0;
    bool ok = true, issued = false, ready = false;
    for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x) {
      const Item it = walk.at(item);
      const uint32_t idesc = idesc_mxf4(128, (it.rows + 15) & ~15);
      const int buf = local % nbuf;
      ok = __all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(kAccEmpty + buf),
                                                 ((uint32_t)(local / nbuf) & 1u) ^ 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * acc_stride;
      for (int kb = 0; kb < a.kblocks; ++kb) {
        if (!ready)
          ok = __all_sync(0xFFFFFFFFu,
                          wait_or_leave(R.bar(kSfReady + stage), phase, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int s = stage;
        const uint32_t sb = smem_u32(stages + s * stage_bytes);
        const uint32_t col = tmem + sf_base + s * slot_cols;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          // the next stage is looked at while this one's first MMAs run
          if (ks == 2)
            ready = __all_sync(0xFFFFFFFFu, phase_done(R.bar(kSfReady + stage), phase));
          const uint32_t id = 2u * (ks & 1);  // which two of a column's four scales
          mma_mxf4_warp(acc, smem_desc(sb + ks * 32, 16, 1024, 2),
                        smem_desc(sb + off_b + ks * 32, 16, 1024, 2),
                        idesc | (id << 4) | (id << 29), col + 4 * (ks >> 1),
                        col + 8 + nrb * (ks >> 1), (kb | ks) != 0 ? 1u : 0u);
        }
        issued = true;
        tc_commit_warp(R.bar(kEmpty + s));
      }
      if (!ok) break;
      tc_commit_warp(R.bar(kAccFull + buf));
      ++local;
    }
    if ((!ok || *abort_flag) && issued) {
      tc_commit_warp(R.bar(kDrain));
      mbar_wait(R.bar(kDrain), 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    using T = typename Elem<DT>::type;
    const int q = warp & 3;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    T* out = static_cast<T*>(a.out);
    int local = 0;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const Item it = walk.at(item);
      const int n = it.mt * 128 + q * 32 + lane;  // this lane's feature
      const int n16 = (it.rows + 15) & ~15;
      const int buf = local % nbuf;
      if (!__all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(kAccFull + buf),
                                                 (uint32_t)(local / nbuf) & 1u, abort_flag))) {
        // what this warp leaves: NaN in its features
        for (; item < n_items; item += gridDim.x) {
          const Item left = walk.at(item);
          const int f = left.mt * 128 + q * 32 + lane;
          for (int j = 0; f < a.N && j < left.rows; ++j)
            out[(left.row0 + j) * a.ld + f] = (T)float_to_elem<DT>(__int_as_float(0x7FC00000));
        }
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + lane_addr + buf * acc_stride;
      for (int c0 = 0; c0 < n16; c0 += 32) {
        const int ncol = min(32, n16 - c0);
        float v[32];
        tmem_ld16(acc + c0, *reinterpret_cast<float(*)[16]>(v));
        if (ncol > 16) tmem_ld16(acc + c0 + 16, *reinterpret_cast<float(*)[16]>(v + 16));
        tmem_wait_ld();
        if (c0 + 32 >= n16) {
          tc_fence_before();
          mbar_arrive(R.bar(kAccEmpty + buf));
        }
        const int m = min(32, it.rows - c0);
        T* o = out + (int64_t)(it.row0 + c0) * a.ld;
        if (DT != kF32 && a.wide) {
          // A 4 x 4 transpose between four lanes, two rounds of exchange: lane i of a quad
          // ends with features f .. f + 3 of row j + i, one store of 8 bytes.
          const bool odd = lane & 1, upper = lane & 2;
          const int f = n & ~3;
          T* p = o + (int64_t)(lane & 3) * a.ld + f;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const uint32_t w01 = pack2<DT>(v[j], v[j + 1]), w23 = pack2<DT>(v[j + 2], v[j + 3]);
            const uint32_t x01 = __shfl_xor_sync(0xFFFFFFFFu, w01, 1);
            const uint32_t x23 = __shfl_xor_sync(0xFFFFFFFFu, w23, 1);
            const uint32_t a01 = odd ? __byte_perm(x01, w01, 0x7632) : __byte_perm(w01, x01, 0x5410);
            const uint32_t a23 = odd ? __byte_perm(x23, w23, 0x7632) : __byte_perm(w23, x23, 0x5410);
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? a01 : a23, 2);
            if (j + (lane & 3) < m && f < a.N)
              *reinterpret_cast<uint2*>(p + j * a.ld) =
                  upper ? make_uint2(got, a23) : make_uint2(a01, got);
          }
        } else if (n < a.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < m) o[j * a.ld + n] = (T)float_to_elem<DT>(v[j]);
        }
      }
      ++local;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- CTA pairs
// The same product where an expert has rows enough to fill the tensor cores: two CTAs of a
// cluster share a tile of 256 weight rows x up to 256 rows (cta_group::2).  Each holds 128
// weight rows, half of the rows' codes and 128 lanes of accumulators, and all the rows'
// scales; rank 0 issues every MMA.  Against single CTAs a stage brings 32 KB for 256 x 256 x
// 256 / 2 products in place of 40 KB for 128 x 192 x 256, and each role's work a stage (some
// 250 to 500 cycles: waits, copies, scales to TMEM, issue) is spread over 512 cycles of MMA
// in place of 384.  256 columns of accumulators leave no room for a second buffer beside the
// scales (192 of them would, twice, and measured 10 to 20 % slower): eight epilogue warps take
// them to registers as 16-bit pairs, free them, and store while the next item's MMAs run.
// Measured: 16384 rows N4096 D7168 on 8 experts 145 us (6.6 PFLOP/s; kind::mxf4 issues 16384
// products a cycle and SM, 9.6 PFLOP/s at 1.92 GHz), on 32 ragged ones 167 us, one matrix of
// 4096 rows 40 us (fp32 results, whose accumulators are held until stored: 203, 224 and 52);
// single CTAs 196, 224 and 60.  A stage's MMAs take 512 of its 550 cycles, the
// pause between items 1850 (drain, then refill); copies bring 65 bytes a cycle and SM, and
// halving the rows' took 6 % off, which sharing them by multicast could gain at most.
namespace pair {
constexpr int kThreads = 512;  // 0 weights, 1 MMA, 2 rows, 3 scales, 4-7 scales to TMEM, 8-15 epilogue
constexpr int kTileN = 256;       // rows of the largest tile
constexpr int kStages = 8;
constexpr int kFull = 0;
constexpr int kEmpty = kStages;
constexpr int kSfReady = 2 * kStages;  // rank 0's: 4 warps of both CTAs
constexpr int kAccFull = 3 * kStages;
constexpr int kAccEmpty = kAccFull + 2;  // rank 0's: 8 warps of both CTAs
constexpr int kDrain = kAccEmpty + 2;
constexpr int kBars = kDrain + 1;
constexpr int kFlagsOff = 8 * kBars;
constexpr int kWarpSumOff = kFlagsOff + 32;
static_assert(kWarpSumOff + 4 * (kThreads / 32) <= kGroupsOff, "barrier area");

__device__ __forceinline__ void alloc(uint32_t slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// Arrive on the barrier at this address in both CTAs once the MMAs so far are done.
__device__ __forceinline__ void commit_warp(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b16 m;\n mov.b16 m, 3;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], m;\n}" ::"r"(bar)
      : "memory");
}
// Arrive on rank 0's barrier, with the instruction's default order (release, this CTA).
// What is handed over lies in TMEM and shared memory, which have one copy, and is complete:
// the caller has waited for its tcgen05.st or tcgen05.ld, and has seen the copies' mbarrier.
// The order of a whole cluster's memory costs some 1000 cycles an arrival, two stages' MMAs.
__device__ __forceinline__ void arrive_rank0(uint32_t bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(r) : "memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
}  // namespace pair

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
    gemm_mx_pair_kernel(const __grid_constant__ MxMaps maps, const __grid_constant__ MxGemmArgs a) {
  using namespace pair;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const Ring R{smem};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + pair::kFlagsOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_most = reinterpret_cast<int*>(tmem_slot + 3);
  int* s_sum = reinterpret_cast<int*>(smem + pair::kWarpSumOff);
  int* first_item = reinterpret_cast<int*>(smem + kGroupsOff);
  int* first_row = first_item + a.E + 1;

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int m_pairs = (a.N + 255) / 256;
  if (threadIdx.x == 0) {
    for (int s = 0; s < pair::kStages; ++s) {
      mbar_init(R.bar(pair::kFull + s), 3);  // weights, rows, scales
      mbar_init(R.bar(pair::kEmpty + s), 1);
      mbar_init(R.bar(pair::kSfReady + s), 8);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(R.bar(pair::kAccFull + b), 1);
      mbar_init(R.bar(pair::kAccEmpty + b), 16);
    }
    mbar_init(R.bar(pair::kDrain), 1);
    *abort_flag = 0;
    *s_most = 32;
    fence_barrier_init();
    prefetch_tmap(&maps.w);
    for (int i = 0; i < 8; ++i) prefetch_tmap(&maps.x[i]);
  }
  __syncwarp();
  if (warp == 1) pair::alloc(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers and TMEM are there
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  pdl_wait();
  pdl_trigger();
  const int item0 = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;
  lay_out_groups<pair::kThreads>(a, a.tile_rows, 32, m_pairs, first_item, first_row, s_sum,
                                 s_most);
  const int n_items = uniform(first_item[a.E]);

  const int most = uniform(*s_most);                // rows of the largest tile, whole 32s
  const int sfb_bytes = (8 * (most + 2) + 127) & ~127;
  const int off_b = kABytes, off_sfa = off_b + most / 2 * kRowBytes, off_sfb = off_sfa + kSfaBytes;
  const int stage_bytes = (off_sfb + sfb_bytes + 1023) & ~1023;
  const int nrb = most <= 128 ? 4 : 8;
  const int slot_cols = 8 + 2 * nrb;
  // two accumulator buffers where they leave room for the scales of five stages
  const int nbuf = 2 * most + 5 * slot_cols <= kTmemCols ? 2 : 1;
  const int sf_base = nbuf * most;             // scales behind the accumulators
  const int head = (kGroupsOff + 8 * (a.E + 1) + 1023) & ~1023;
  uint8_t* stages = smem + head;
  const int n_stages = min(min(pair::kStages, (kSmem - 1024 - head) / stage_bytes),
                           (kTmemCols - sf_base) / slot_cols);

  Walk walk{first_item, first_row, m_pairs, 32, 0};
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&] {
    if (++stage == n_stages) {
      stage = 0;
      phase ^= 1;
    }
  };
  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ producers
    const uint64_t pol = policy_evict_last();
    const int64_t w_rows = ((int64_t)a.E * a.N + 1) & ~int64_t(1);
    const int x_rows = (a.R + 1) & ~1;
    int loaded = 0;
    bool ok = true;
    for (int item = item0; ok && item < n_items; item += step) {
      if (warp == 2 && item == a.leave_item) break;
      const Item it = walk.at(item);
      const int half = ((it.rows + 31) & ~31) / 2;
      const int x0 = it.row0 + rank * half;
      // a tile's last 128 weight rows may lie past the last weight: then no box is needed, but
      // one of rows that exist keeps every stage alike
      const int64_t w0 = min((int64_t)it.e * a.N + it.mt * 256 + rank * 128,
                             (int64_t)a.E * a.N - 1);
      const int64_t w_even = w0 & ~int64_t(1);
      const int x_even = it.row0 & ~1;
      const uint32_t sfa = 8u * (uint32_t)min((int64_t)(w0 != w_even ? 130 : 128), w_rows - w_even);
      const uint32_t sfb = 8u * (uint32_t)min(2 * half + (it.row0 != x_even ? 2 : 0), x_rows - x_even);
      for (int kb = 0; kb < a.kblocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu,
                        wait_or_leave(R.bar(pair::kEmpty + stage), phase ^ 1, abort_flag));
        if (!ok) break;
        const uint32_t sb = smem_u32(stages + stage * stage_bytes);
        const uint32_t full = R.bar(pair::kFull + stage);
        if (warp == 0) {
          expect_warp(full, kABytes);
          box_warp(sb, &maps.w, full, kb * kRowBytes, (int)w0, pol);
        } else if (warp == 2) {
          expect_warp(full, half * kRowBytes);
          box_warp(sb + off_b, &maps.x[half / 16 - 1], full, kb * kRowBytes, x0, pol);
        } else {
          expect_warp(full, sfa + sfb);
          piece_warp(sb + off_sfa, a.sw + kb * a.sw_panel + 8 * w_even, sfa, full);
          piece_warp(sb + off_sfb, a.sx + kb * a.sx_panel + 8 * (int64_t)x_even, sfb, full);
        }
        ++loaded;
        advance();
      }
    }
    if (ok && warp == 0) await_ring(R, pair::kEmpty, loaded, n_stages, abort_flag);
    if (!ok || *abort_flag) drain_ring(R, loaded, n_stages);
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ scales to TMEM
    const uint32_t lane_q = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = true;
    for (int item = item0; ok && item < n_items; item += step) {
      const Item it = walk.at(item);
      const int64_t w0 = min((int64_t)it.e * a.N + it.mt * 256 + rank * 128,
                             (int64_t)a.E * a.N - 1);
      const int odd_w = (int)(w0 & 1), odd_x = it.row0 & 1;
      for (int kb = 0; kb < a.kblocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, wait_or_leave(R.bar(pair::kFull + stage), phase, abort_flag));
        if (!ok) break;
        tc_fence_after();  // as the single CTAs
        const uint32_t sb = smem_u32(stages + stage * stage_bytes);
        const uint32_t col = tmem + lane_q + sf_base + stage * slot_cols;
        const uint32_t sa = sb + off_sfa + 8 * (odd_w + lane), sx = sb + off_sfb + 8 * (odd_x + lane);
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 p = lds64(sa + 256 * j);
          v[j] = p.x, v[4 + j] = p.y;
        }
        pair::st8(col, v);
        if (nrb == 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint2 p = 32 * j < it.rows ? lds64(sx + 256 * j) : make_uint2(0u, 0u);
            v[j] = p.x, v[4 + j] = p.y;
          }
          pair::st8(col + 8, v);
        } else {
          uint32_t u[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint2 p = 32 * j < it.rows ? lds64(sx + 256 * j) : make_uint2(0u, 0u);
            u[j] = p.x, u[8 + j] = p.y;
          }
          tmem_st16(col + 8, u);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_rank0(R.bar(pair::kSfReady + stage));
        advance();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (rank 0)
    bool ok = rank == 0, issued = false, ready = false;
    int local = 0;
    for (int item = item0; ok && item < n_items; item += step, ++local) {
      const Item it = walk.at(item);
      const uint32_t idesc = idesc_mxf4(256, (it.rows + 31) & ~31);
      const int buf = nbuf == 2 ? local & 1 : 0;
      const uint32_t acc_par = ((uint32_t)(nbuf == 2 ? local >> 1 : local) & 1u) ^ 1u;
      ok = __all_sync(0xFFFFFFFFu,
                      wait_or_leave(R.bar(pair::kAccEmpty + buf), acc_par, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * most;
      for (int kb = 0; kb < a.kblocks; ++kb) {
        if (!ready)
          ok = __all_sync(0xFFFFFFFFu,
                          wait_or_leave(R.bar(pair::kSfReady + stage), phase, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const int s = stage;
        const uint32_t sb = smem_u32(stages + s * stage_bytes);
        const uint32_t col = tmem + sf_base + s * slot_cols;
        advance();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (ks == 2)
            ready = __all_sync(0xFFFFFFFFu, phase_done(R.bar(pair::kSfReady + stage), phase));
          const uint32_t id = 2u * (ks & 1);
          pair::mma_warp(acc, smem_desc(sb + ks * 32, 16, 1024, 2),
                         smem_desc(sb + off_b + ks * 32, 16, 1024, 2),
                         idesc | (id << 4) | (id << 29), col + 4 * (ks >> 1),
                         col + 8 + nrb * (ks >> 1), (kb | ks) != 0 ? 1u : 0u);
        }
        issued = true;
        pair::commit_warp(R.bar(pair::kEmpty + s));
      }
      if (!ok) break;
      pair::commit_warp(R.bar(pair::kAccFull + buf));
    }
    if (issued && (!ok || *abort_flag)) {
      pair::commit_warp(R.bar(pair::kDrain));
      mbar_wait(R.bar(pair::kDrain), 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    using T = typename Elem<DT>::type;
    const int q = warp & 3, h = (warp - 8) >> 2;  // lanes 32q ..., first or second half of the rows
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    T* out = static_cast<T*>(a.out);
    int local = 0;
    for (int item = item0; item < n_items; item += step, ++local) {
      const Item it = walk.at(item);
      const int n = it.mt * 256 + rank * 128 + q * 32 + lane;
      const int half = ((it.rows + 31) & ~31) / 2;
      const int buf = nbuf == 2 ? local & 1 : 0;
      const uint32_t acc_par = (uint32_t)(nbuf == 2 ? local >> 1 : local) & 1u;
      if (!__all_sync(0xFFFFFFFFu,
                      wait_or_leave(R.bar(pair::kAccFull + buf), acc_par, abort_flag))) {
        for (; item < n_items; item += step) {
          const Item left = walk.at(item);
          const int f = left.mt * 256 + rank * 128 + q * 32 + lane;
          for (int j = h; f < a.N && j < left.rows; j += 2)
            out[(left.row0 + j) * a.ld + f] = (T)float_to_elem<DT>(__int_as_float(0x7FC00000));
        }
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + lane_addr + buf * most + h * half;
      const int m = min(half, it.rows - h * half);  // rows of this half
      T* o = out + (int64_t)(it.row0 + h * half) * a.ld;
      if constexpr (DT != kF32) {
        uint32_t w[64];  // 128 rows in pairs
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // two loads of 16 columns in flight
          if (32 * g >= half) continue;
          float v[32];
          tmem_ld16(acc + 32 * g, *reinterpret_cast<float(*)[16]>(v));
          if (32 * g + 16 < half)
            tmem_ld16(acc + 32 * g + 16, *reinterpret_cast<float(*)[16]>(v + 16));
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) w[16 * g + i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_rank0(R.bar(pair::kAccEmpty + buf));
        if (a.wide) {
          // the 4 x 4 exchange of the single CTAs
          const bool odd = lane & 1, upper = lane & 2;
          const int f = n & ~3;
          T* p = o + (int64_t)(lane & 3) * a.ld + f;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (16 * g >= half) break;  // a branch for 16 rows: their exchanges overlap
#pragma unroll
            for (int j = 16 * g; j < 16 * g + 16; j += 4) {
              const uint32_t w01 = w[j / 2], w23 = w[j / 2 + 1];
              const uint32_t x01 = __shfl_xor_sync(0xFFFFFFFFu, w01, 1);
              const uint32_t x23 = __shfl_xor_sync(0xFFFFFFFFu, w23, 1);
              const uint32_t a01 = odd ? __byte_perm(x01, w01, 0x7632) : __byte_perm(w01, x01, 0x5410);
              const uint32_t a23 = odd ? __byte_perm(x23, w23, 0x7632) : __byte_perm(w23, x23, 0x5410);
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? a01 : a23, 2);
              if (j + (lane & 3) < m && f < a.N)
                *reinterpret_cast<uint2*>(p) = upper ? make_uint2(got, a23) : make_uint2(a01, got);
              p += 4 * a.ld;
            }
          }
        } else if (n < a.N) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j < m) o[j * a.ld + n] = (T)(w[j / 2] >> (16 * (j & 1)));
        }
      } else {
        for (int c = 0; c < half; c += 16) {
          float v[16];
          tmem_ld16(acc + c, v);
          tmem_wait_ld();
          if (n < a.N)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < m) o[(c + j) * a.ld + n] = (T)float_to_elem<DT>(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_rank0(R.bar(pair::kAccEmpty + buf));
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // neither CTA's shared memory or TMEM is used any more
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    pair::dealloc(tmem, kTmemCols);
  }
}

bool use_pairs(const MxGemmArgs& a, int sms) {
  const int64_t items = (int64_t)a.R / pair::kTileN * ((a.N + 255) / 256);
  return a.N > 128 && a.kblocks >= kPairStages && a.R >= a.E * kPairRows && items >= sms / 4;
}

// Rows of the largest tile of pairs: 256; of a single matrix less where the items then come
// out in fuller rounds of the pairs.  A stage of an item takes some 316 + rows cycles.  R4096
// N4096 D7168 by 76 pairs: 256 items are 4 rounds, the last a third full, and so are 304 items
// of 224 rows (41.7 -> 40.0 us); R8192 stays at 256.
int tile_rows(const MxGemmArgs& a, int pairs) {
  int best = pair::kTileN;
  int64_t best_cost = INT64_MAX;
  for (int h = pair::kTileN; h >= 192 && !a.offsets; h -= 32) {
    const int64_t items = (int64_t)((a.R + h - 1) / h) * ((a.N + 255) / 256);
    const int64_t cost = (items + pairs - 1) / pairs * (316 + h);
    if (cost < best_cost) best = h, best_cost = cost;
  }
  return best;
}

template <typename K>
cudaError_t launch_kernel(K kernel, int threads, std::atomic<uint64_t>& configured,
                          const MxMaps& maps, const MxGemmArgs& a, int grid, cudaStream_t s) {
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(grid), dim3(threads), (size_t)kSmem, s, maps, a);
}

template <int DT>
cudaError_t launch_typed(const MxMaps& maps, const MxGemmArgs& a, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> single_set{0}, pair_set{0};
  if (use_pairs(a, sms)) {
    MxGemmArgs p = a;
    p.tile_rows = tile_rows(a, sms / 2);
    const int64_t tiles = (int64_t)a.R / p.tile_rows + a.E;
    const int64_t pairs = std::min<int64_t>(sms / 2, tiles * ((a.N + 255) / 256));
    return launch_kernel(gemm_mx_pair_kernel<DT>, pair::kThreads, pair_set, maps, p,
                         (int)pairs * 2, s);
  }
  const int64_t tiles = std::min<int64_t>(a.R, (int64_t)a.R / kTileN + a.E);
  const int grid = (int)std::min<int64_t>(sms, tiles * ((a.N + 127) / 128));
  return launch_kernel(gemm_mx_kernel<DT>, kThreads, single_set, maps, a, grid, s);
}

}  // namespace

cudaError_t launch_gemm_mx(const MxGemmArgs& a, const uint8_t* x_codes, const uint8_t* w_codes,
                           int sms, cudaStream_t s) {
  MxMaps maps;
  const uint64_t row_bytes = (uint64_t)a.kblocks * kRowBytes;
  if (!byte_map(&maps.w, w_codes, row_bytes, (uint64_t)a.E * a.N, 128)) return cudaErrorInvalidValue;
  for (int i = 0; i < 8; ++i)
    if (!byte_map(&maps.x[i], x_codes, row_bytes, a.R, 16u * (i + 1))) return cudaErrorInvalidValue;
  return a.dtype == kF32    ? launch_typed<kF32>(maps, a, sms, s)
         : a.dtype == kBf16 ? launch_typed<kBf16>(maps, a, sms, s)
                            : launch_typed<kF16>(maps, a, sms, s);
}

}  // namespace moe
