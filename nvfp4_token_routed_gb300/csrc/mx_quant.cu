// mx_quant.cu -- microscaled FP4: rows to E2M1 codes with one power of two per 32 values
// (block32.cuh), and back.
//
// Codes lie as the rows do, two to a byte, a row padded with zeros to a multiple of 256
// values (one stage of the product).  Scales lie in panels: the 8 bytes of a row's 256
// values, rows one after the other, panel after panel, the number of rows rounded up to
// even.  So the scales that a stage of the product needs for any run of consecutive rows
// are one contiguous piece, which one bulk copy brings, and a run of rows may start at any
// row: experts' groups need no padding.
//
// A warp takes 256 values of a row, 8 a lane, four such spans where there are rows enough
// (one: 80 us, four: 53; maxima of 16-bit halves two at a time: 48).  Measured (bf16, 16384 x
// 7168; copy rate 6686 GB/s): 48 us, 0.94 of the copy rate, with 75 % of the issue slots used.
// Rows off 16 bytes gain as much: 3719 x 6662 in one span a warp 17.5 us, in four 12.6.
#include "block32.cuh"
#include "experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
static_assert(kMxPanel == kSpan, "a panel is a warp's span");

template <int DT, int VB>
__device__ __forceinline__ void* warp_stage() {
  __shared__ __align__(16) uint8_t stage[kThreads / 32][kSpanBytes<DT, VB>];
  return stage[threadIdx.x >> 5];
}

// A warp's 256 values (lane l holds 8l ... 8l+7): 4 bytes of codes a lane, 8 of scales.
template <int DT>
__device__ __forceinline__ void write_panel(const MxQuantArgs& a, int64_t r, int panel,
                                            const uint32_t (&w)[kRunWords<DT>]) {
  const int lane = threadIdx.x & 31;
  const uint32_t byte = block_scale_byte<E2m1>(block_amax<DT>(w));
  Run8 v;
  run_unpack<DT>(w, v);
  reinterpret_cast<uint32_t*>(a.codes + r * (a.Dp / 2) + panel * (kMxPanel / 2))[lane] =
      byte == 255u ? 0u : e2m1x8(v, block_inverse(byte));
  // lane 4b holds block b's byte; lanes 0 and 16 gather four each
  uint32_t lo = byte | (__shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8);
  lo |= __shfl_down_sync(0xFFFFFFFFu, lo, 8) << 16;
  const uint32_t hi = __shfl_sync(0xFFFFFFFFu, lo, 16);
  const int64_t rows_p = ((int64_t)a.R + 1) & ~int64_t(1);
  if (lane == 0)
    *reinterpret_cast<uint2*>(a.scales + (panel * rows_p + r) * 8) = make_uint2(lo, hi);
}

// A warp's row and first of U panels; false: nothing to do.
__device__ __forceinline__ bool place_of(const MxQuantArgs& a, int segs, int u, int64_t& r,
                                         int& panel) {
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  r = i <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / (uint32_t)segs) : i / segs;
  panel = (int)(i - r * segs) * u;
  return r < (a.n_rows ? min(a.R, *a.n_rows) : a.R);
}

// U panels a warp, their loads issued together.
template <int DT, int VB, int U>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const MxQuantArgs a, int segs) {
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int panel;
  if (!place_of(a, segs, U, r, panel)) return;
  void* stage = warp_stage<DT, VB>();
  const int c = panel * kMxPanel;
  const auto* x = static_cast<const typename Elem<DT>::type*>(a.x) + r * a.ld_x + c;
  Span<DT, VB> t[U];
#pragma unroll
  for (int u = 0; u < U; ++u) t[u].load(x + u * kMxPanel, a.D - c - u * kMxPanel);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (U > 1 && (panel + u) * kMxPanel >= a.Dp) break;
    uint32_t w[kRunWords<DT>];
    t[u].runs(stage, w);
    write_panel<DT>(a, r, panel + u, w);
  }
}

template <int DT, int VB, int U>
__global__ void __launch_bounds__(kThreads) restore_kernel(const MxQuantArgs a, int segs) {
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int panel;
  if (!place_of(a, segs, U, r, panel)) return;
  const int lane = threadIdx.x & 31, c = panel * kMxPanel;
  const int64_t rows_p = ((int64_t)a.R + 1) & ~int64_t(1);
  uint32_t code[U], byte[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    code[u] = byte[u] = 0;
    if (U > 1 && (panel + u) * kMxPanel >= a.Dp) continue;
    code[u] = reinterpret_cast<const uint32_t*>(a.codes + r * (a.Dp / 2) +
                                                (panel + u) * (kMxPanel / 2))[lane];
    byte[u] = a.scales[((panel + u) * rows_p + r) * 8 + (lane >> 2)];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Run8 v;
    e2m1x8_to_float(code[u], block_scale(byte[u]), v);
    span_store<DT, VB>(
        static_cast<typename Elem<DT>::type*>(a.out) + r * a.ld_out + c + u * kMxPanel,
        a.D - c - u * kMxPanel, warp_stage<DT, VB>(), v);
  }
}

// Columns of a stack of matrices as rows: 256 values of 32 columns a block, through
// shared memory (a column's stride of 261 words keeps a warp's reads of 8 consecutive
// values at most 8 to a bank, and its writes free of conflicts).  8 x 4096 x 7168 bf16 in 337
// us, 0.26 of the copy rate, against 94 for the same stack row by row: loads of 2 bytes a lane
// and those conflicts.  It runs once for a layer's weights.
constexpr int kColsT = 32, kStrideT = kMxPanel + 5;
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_t_kernel(const MxQuantArgs a, int C) {
  __shared__ float tile[kColsT * kStrideT];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kColsT, panel = blockIdx.y;
  const int64_t b = blockIdx.z;
  const auto* x = static_cast<const typename Elem<DT>::type*>(a.x) + b * a.D * C;
  for (int j = warp; j < kMxPanel; j += kThreads / 32) {
    const int d = panel * kMxPanel + j;
    tile[lane * kStrideT + j] =
        d < a.D && c0 + lane < C ? elem_to_float<DT>(x[(int64_t)d * C + c0 + lane]) : 0.0f;
  }
  __syncthreads();
  for (int j = warp; j < kColsT && c0 + j < C; j += kThreads / 32) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(tile[j * kStrideT + lane * 8 + i]);
    write_panel<kF32>(a, b * C + c0 + j, panel, w);
  }
}

int size_of(int dtype) { return dtype == kF32 ? 4 : 2; }

template <typename K>
cudaError_t go(K kernel, const MxQuantArgs& a, int u, cudaStream_t s) {
  const int segs = (a.Dp / kMxPanel + u - 1) / u;
  const int64_t blocks = ((int64_t)a.R * segs + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, segs);
}

// U panels a warp where that leaves the device enough warps.  Restored fp32 rows take two:
// 5001 x 1407 5.9 us (by four 6.6, by one 6.6), 20000 x 3001 43 (43, 50), 4096 x 7168 28.5 (30.1,
// 26.1).
template <int U = 4, typename K>
cudaError_t go_many(K one, K many, const MxQuantArgs& a, cudaStream_t s) {
  return (int64_t)a.R * (a.Dp / kMxPanel) >= 4 * 152 * 16 ? go(many, a, U, s) : go(one, a, 1, s);
}
template <int DT>
cudaError_t quantize_typed(const MxQuantArgs& a, cudaStream_t s) {
  switch (access_bytes(a.x, a.ld_x * size_of(DT), (int64_t)a.D * size_of(DT))) {
    case 16: return go_many(quantize_kernel<DT, 16, 1>, quantize_kernel<DT, 16, 4>, a, s);
    case 8: return go_many(quantize_kernel<DT, 8, 1>, quantize_kernel<DT, 8, 4>, a, s);
    case 4: return go_many(quantize_kernel<DT, 4, 1>, quantize_kernel<DT, 4, 4>, a, s);
    default: break;
  }
  if constexpr (DT != kF32)
    return go_many(quantize_kernel<DT, 2, 1>, quantize_kernel<DT, 2, 4>, a, s);
  return cudaErrorInvalidValue;
}
template <int DT>
cudaError_t restore_typed(const MxQuantArgs& a, cudaStream_t s) {
  constexpr int kMany = DT == kF32 ? 2 : 4;
  switch (access_bytes(a.out, a.ld_out * size_of(DT), (int64_t)a.D * size_of(DT))) {
    case 16: return go_many<kMany>(restore_kernel<DT, 16, 1>, restore_kernel<DT, 16, kMany>, a, s);
    case 8: return go_many<kMany>(restore_kernel<DT, 8, 1>, restore_kernel<DT, 8, kMany>, a, s);
    case 4: return go_many<kMany>(restore_kernel<DT, 4, 1>, restore_kernel<DT, 4, kMany>, a, s);
    default: break;
  }
  if constexpr (DT != kF32)
    return go_many<kMany>(restore_kernel<DT, 2, 1>, restore_kernel<DT, 2, kMany>, a, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? quantize_typed<kF32>(a, s)
         : dtype == kBf16 ? quantize_typed<kBf16>(a, s)
                          : quantize_typed<kF16>(a, s);
}
cudaError_t launch_mx_restore(const MxQuantArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? restore_typed<kF32>(a, s)
         : dtype == kBf16 ? restore_typed<kBf16>(a, s)
                          : restore_typed<kF16>(a, s);
}
cudaError_t launch_mx_quantize_t(const MxQuantArgs& a, int C, int dtype, cudaStream_t s) {
  const dim3 grid((C + kColsT - 1) / kColsT, a.Dp / kMxPanel, a.R / C);
  return dtype == kF32
             ? launch_pdl(quantize_t_kernel<kF32>, grid, dim3(kThreads), 0, s, a, C)
         : dtype == kBf16
             ? launch_pdl(quantize_t_kernel<kBf16>, grid, dim3(kThreads), 0, s, a, C)
             : launch_pdl(quantize_t_kernel<kF16>, grid, dim3(kThreads), 0, s, a, C);
}

}  // namespace moe
