// checkpoint.cu -- rows kept in 8 bits, and the experts' activation whose backward pass
// reads them.
//
// Kept: E4M3 in blocks of 32 along the row, a power of two a block (block32.cuh): 8.25
// bits a value in place of 16 or 32.  SwiGLU's gate and up halves are blocked apart, and
// each half's codes are padded with zeros to whole blocks, so that codes lie on 32 bytes
// whatever the width.
//   swiglu   y = g s(g) u, s(g) = 1 / (1 + exp(-g)); with a limit L: g = min(g, L),
//            u = min(max(u, -L), L) first
//            dg = dy u s(g) (1 + g (1 - s(g))) where g <= L, du = dy g s(g) where |u| <= L
//   relu2    y = max(h, 0)^2, dh = 2 dy max(h, 0)
// y comes from the unrounded input, the gradient from the kept values.
//
// A thread takes a run of 8 values (of both halves), four lanes a block; nothing is
// shared between blocks, so the kernels are bound by HBM.
#include <algorithm>

#include "block32.cuh"
#include "experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// A thread's run: row, first value, and how many of its 8 values the row has.
struct Place {
  int64_t r;
  int c;
  int n;       // <= 0: padding of the last block
  bool live;   // the row counts
};
__device__ __forceinline__ Place place_of(const KeepArgs& a, int64_t i, int runs) {
  Place p;
  p.r = i <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / (uint32_t)runs) : i / runs;
  p.c = (int)(i - p.r * runs) * 8;
  const int rows = a.n_rows ? min(a.R, *a.n_rows) : a.R;
  p.live = p.r < rows;
  p.n = p.live ? a.W - p.c : 0;
  return p;
}

// Writes a run's codes and its block's scale.  All lanes take part.
__device__ __forceinline__ void keep_run(const KeepArgs& a, const Place& p, int halves, int half,
                                         const Run8& r) {
  const int Wp = (a.W + 31) & ~31;
  const uint32_t byte = block_scale_byte<E4m3>(quad_max(r.amax_bits()));
  if (!p.live) return;
  const int64_t at = (p.r * halves + half) * Wp + p.c;
  *reinterpret_cast<uint2*>(a.codes + at) =
      byte == 255u ? make_uint2(0u, 0u) : e4m3x8(r, block_inverse(byte));
  if ((threadIdx.x & 3) == 0) a.scales[at >> 5] = (uint8_t)byte;
}
__device__ __forceinline__ void kept_run(const KeepArgs& a, const Place& p, int halves, int half,
                                         Run8& r) {
  const int Wp = (a.W + 31) & ~31;
  const int64_t at = (p.r * halves + half) * Wp + p.c;
  e4m3x8_to_float(*reinterpret_cast<const uint2*>(a.codes + at), block_scale(a.scales[at >> 5]), r);
}

template <int DT>
__device__ __forceinline__ const void* elem_ptr(const void* p, int64_t i) {
  return static_cast<const typename Elem<DT>::type*>(p) + i;
}
template <int DT>
__device__ __forceinline__ void* elem_ptr(void* p, int64_t i) {
  return static_cast<typename Elem<DT>::type*>(p) + i;
}

template <int DT, int VB>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(const KeepArgs a, int runs) {
  pdl_trigger();
  pdl_wait();
  const Place p = place_of(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, runs);
  uint32_t w[kRunWords<DT>];
  run_load_raw<DT, VB>(elem_ptr<DT>(a.x, p.r * a.ld_x + p.c), p.n, w);
  Run8 r;
  run_unpack<DT>(w, r);
  keep_run(a, p, 1, 0, r);
}

template <int DT, int VB>
__global__ void __launch_bounds__(kThreads) restore_kernel(const KeepArgs a, int runs) {
  pdl_trigger();
  pdl_wait();
  const Place p = place_of(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, runs);
  if (p.n <= 0) return;
  Run8 r;
  kept_run(a, p, 1, 0, r);
  run_store<DT, VB>(elem_ptr<DT>(a.out, p.r * a.ld_out + p.c), p.n, r);
}

// s(g): correctly to fp32's last bits for fp32 rows, by the fast exponential (2^-21 of
// the result) where y is rounded to 16 bits.
template <int DT>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (DT == kF32) return 1.0f / (1.0f + expf(-g));
  return __fdividef(1.0f, 1.0f + __expf(-g));
}
// Comparisons, not fminf: a NaN stays one.
__device__ __forceinline__ float cap(float g, float L) { return g > L ? L : g; }
__device__ __forceinline__ float clip(float u, float L) { return u > L ? L : u < -L ? -L : u; }

template <int DT, int VB, int ACT>
__global__ void __launch_bounds__(kThreads) act_kernel(const KeepArgs a, int runs) {
  pdl_trigger();
  pdl_wait();
  const Place p = place_of(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, runs);
  uint32_t wg[kRunWords<DT>], wu[kRunWords<DT>];
  run_load_raw<DT, VB>(elem_ptr<DT>(a.x, p.r * a.ld_x + p.c), p.n, wg);
  if (ACT == kActSwiglu) run_load_raw<DT, VB>(elem_ptr<DT>(a.x, p.r * a.ld_x + a.W + p.c), p.n, wu);
  Run8 g, u, y;
  run_unpack<DT>(wg, g);
  if (ACT == kActSwiglu) {
    run_unpack<DT>(wu, u);
    const float L = a.limit > 0.0f ? a.limit : __int_as_float(0x7F800000);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gc = cap(g.v[i], L);
      y.v[i] = gc * sigmoid<DT>(gc) * clip(u.v[i], L);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = g.v[i] < 0.0f ? 0.0f : g.v[i];
      y.v[i] = h * h;
    }
  }
  run_store<DT, VB>(elem_ptr<DT>(a.out, p.r * a.ld_out + p.c), p.n, y);
  if (!a.codes) return;
  constexpr int kHalves = ACT == kActSwiglu ? 2 : 1;
  keep_run(a, p, kHalves, 0, g);
  if (ACT == kActSwiglu) keep_run(a, p, kHalves, 1, u);
}

template <int DT, int VB, int ACT>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const KeepArgs a, int runs) {
  pdl_trigger();
  pdl_wait();
  const Place p = place_of(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, runs);
  if (p.n <= 0) return;
  uint32_t wd[kRunWords<DT>];
  run_load_raw<DT, VB>(elem_ptr<DT>(a.x, p.r * a.ld_x + p.c), p.n, wd);
  constexpr int kHalves = ACT == kActSwiglu ? 2 : 1;
  Run8 g, u, d;
  kept_run(a, p, kHalves, 0, g);
  if (ACT == kActSwiglu) kept_run(a, p, kHalves, 1, u);
  run_unpack<DT>(wd, d);
  if (ACT == kActSwiglu) {
    const float L = a.limit > 0.0f ? a.limit : __int_as_float(0x7F800000);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gk = g.v[i], uk = u.v[i];
      const float gc = cap(gk, L), uc = clip(uk, L), s = sigmoid<DT>(gc);
      g.v[i] = gk > L ? 0.0f : d.v[i] * uc * (s * (1.0f + gc * (1.0f - s)));
      u.v[i] = fabsf(uk) > L ? 0.0f : d.v[i] * (gc * s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g.v[i] = 2.0f * d.v[i] * (g.v[i] < 0.0f ? 0.0f : g.v[i]);
  }
  run_store<DT, VB>(elem_ptr<DT>(a.out, p.r * a.ld_out + p.c), p.n, g);
  if (ACT == kActSwiglu)
    run_store<DT, VB>(elem_ptr<DT>(a.out, p.r * a.ld_out + a.W + p.c), p.n, u);
}

int size_of(int dtype) { return dtype == kF32 ? 4 : 2; }

// Widest access to rows of W values, the second half W values further on.
int width(const void* p, int64_t ld, int W, int dtype) {
  return access_bytes(p, ld * size_of(dtype), (int64_t)W * size_of(dtype));
}

template <typename K>
cudaError_t go(K kernel, const KeepArgs& a, cudaStream_t s) {
  const int runs = (a.W + 31) / 32 * 4;
  const int64_t blocks = ((int64_t)a.R * runs + kThreads - 1) / kThreads;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, runs);
}

#define MOE_BY_WIDTH(KERNEL, DT, vb, ...)                                   \
  switch (vb) {                                                             \
    case 16: return go(KERNEL<DT, 16 __VA_ARGS__>, a, s);                   \
    case 8: return go(KERNEL<DT, 8 __VA_ARGS__>, a, s);                     \
    case 4: return go(KERNEL<DT, 4 __VA_ARGS__>, a, s);                     \
    default: break;                                                         \
  }                                                                         \
  if constexpr (DT != kF32) return go(KERNEL<DT, 2 __VA_ARGS__>, a, s);     \
  return cudaErrorInvalidValue;
#define MOE_COMMA ,

template <int DT>
cudaError_t checkpoint_typed(const KeepArgs& a, cudaStream_t s) {
  MOE_BY_WIDTH(checkpoint_kernel, DT, width(a.x, a.ld_x, a.W, DT))
}
template <int DT>
cudaError_t restore_typed(const KeepArgs& a, cudaStream_t s) {
  MOE_BY_WIDTH(restore_kernel, DT, width(a.out, a.ld_out, a.W, DT))
}
template <int DT, int ACT>
cudaError_t act_typed(const KeepArgs& a, cudaStream_t s) {
  const int vb = std::min(width(a.x, a.ld_x, a.W, DT), width(a.out, a.ld_out, a.W, DT));
  MOE_BY_WIDTH(act_kernel, DT, vb, MOE_COMMA ACT)
}
template <int DT, int ACT>
cudaError_t act_grad_typed(const KeepArgs& a, cudaStream_t s) {
  const int vb = std::min(width(a.x, a.ld_x, a.W, DT), width(a.out, a.ld_out, a.W, DT));
  MOE_BY_WIDTH(act_grad_kernel, DT, vb, MOE_COMMA ACT)
}
#undef MOE_BY_WIDTH
#undef MOE_COMMA

}  // namespace

cudaError_t launch_checkpoint(const KeepArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? checkpoint_typed<kF32>(a, s)
         : dtype == kBf16 ? checkpoint_typed<kBf16>(a, s)
                          : checkpoint_typed<kF16>(a, s);
}
cudaError_t launch_restore(const KeepArgs& a, int dtype, cudaStream_t s) {
  return dtype == kF32    ? restore_typed<kF32>(a, s)
         : dtype == kBf16 ? restore_typed<kBf16>(a, s)
                          : restore_typed<kF16>(a, s);
}
cudaError_t launch_expert_act(const KeepArgs& a, int act, int dtype, cudaStream_t s) {
  if (act == kActSwiglu)
    return dtype == kF32    ? act_typed<kF32, kActSwiglu>(a, s)
           : dtype == kBf16 ? act_typed<kBf16, kActSwiglu>(a, s)
                            : act_typed<kF16, kActSwiglu>(a, s);
  return dtype == kF32    ? act_typed<kF32, kActRelu2>(a, s)
         : dtype == kBf16 ? act_typed<kBf16, kActRelu2>(a, s)
                          : act_typed<kF16, kActRelu2>(a, s);
}
cudaError_t launch_expert_act_grad(const KeepArgs& a, int act, int dtype, cudaStream_t s) {
  if (act == kActSwiglu)
    return dtype == kF32    ? act_grad_typed<kF32, kActSwiglu>(a, s)
           : dtype == kBf16 ? act_grad_typed<kBf16, kActSwiglu>(a, s)
                            : act_grad_typed<kF16, kActSwiglu>(a, s);
  return dtype == kF32    ? act_grad_typed<kF32, kActRelu2>(a, s)
         : dtype == kBf16 ? act_grad_typed<kBf16, kActRelu2>(a, s)
                          : act_grad_typed<kF16, kActRelu2>(a, s);
}

}  // namespace moe
