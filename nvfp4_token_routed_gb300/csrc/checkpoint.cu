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
// A warp takes U times 256 consecutive values of a row (of both halves), 8 a lane and four
// lanes a block of 32; its loads are issued together (U = 1: clamped SwiGLU 86 us, 2: 75).
// Nothing is shared between blocks: the kernels are bound by HBM once the instructions fit
// beside it, for which 16-bit maxima and fp32 arithmetic go two at a time (75 -> 61 us).
// Measured (bf16; copy rate 6686 GB/s): clamped SwiGLU 24576 x 2048 forward 61 us (0.99 of the
// copy rate), gradient 65 us (0.93), rows of 4096 x 7168 kept 13.6 us and restored 12.5 us;
// squared ReLU 5001 x 1407 f16, rows off 4 bytes, 16.7 us for both (by a run a lane 31); rows
// off 16 bytes of 3719 x 6662 kept 12.2 us (L2 warm; one span a warp 17.1) and restored 10.2
// (15.4).
#include <algorithm>

#include "block32.cuh"
#include "experts.h"
#include "internal.h"
#include "logits.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// A warp's stage for spans of rows that do not lie on 16 bytes.
template <int DT, int VB>
__device__ __forceinline__ void* warp_stage() {
  __shared__ __align__(16) uint8_t stage[kThreads / 32][kSpanBytes<DT, VB>];
  return stage[threadIdx.x >> 5];
}

// A warp's row and its first span's first value; false: nothing to do.
__device__ __forceinline__ bool place_of(const KeepArgs& a, int segs, int u, int64_t& r, int& c) {
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  r = i <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / (uint32_t)segs) : i / segs;
  c = (int)(i - r * segs) * (u * kSpan);
  return r < (a.n_rows ? min(a.R, *a.n_rows) : a.R);
}

// Writes a run's codes and its block's scale; c: the span's first value.  All lanes take
// part.
template <int DT>
__device__ __forceinline__ void keep_run(const KeepArgs& a, int64_t r, int c, int halves, int half,
                                         const uint32_t (&w)[kRunWords<DT>], Run8& v) {
  const int Wp = (a.W + 31) & ~31;
  c += (threadIdx.x & 31) * 8;
  const uint32_t byte = block_scale_byte<E4m3>(block_amax<DT>(w));
  if (c >= Wp) return;
  // from 248 2^e on a value rounds to 256 2^e: where the type ends before that it takes 240 2^e,
  // which is still within 2^-4 of it, and not an infinity
  constexpr uint32_t kLastByte = DT == kF16 ? 8 + 127 : 120 + 127;
  if (byte == kLastByte) {
    const float most = 240.0f * block_scale(kLastByte);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = fminf(fmaxf(v.v[i], -most), most);
  }
  const int64_t at = (r * halves + half) * Wp + c;
  *reinterpret_cast<uint2*>(a.codes + at) =
      byte == 255u ? make_uint2(0u, 0u) : e4m3x8(v, block_inverse(byte));
  if ((threadIdx.x & 3) == 0) a.scales[at >> 5] = (uint8_t)byte;
}
// A run's codes and scale byte, zeros past the row.
struct Kept {
  uint2 codes;
  uint32_t byte;
};
__device__ __forceinline__ Kept kept_run(const KeepArgs& a, int64_t r, int c, int halves,
                                         int half) {
  const int Wp = (a.W + 31) & ~31;
  c += (threadIdx.x & 31) * 8;
  if (c >= a.W) return Kept{make_uint2(0u, 0u), 0u};
  const int64_t at = (r * halves + half) * Wp + c;
  return Kept{*reinterpret_cast<const uint2*>(a.codes + at), a.scales[at >> 5]};
}

template <int DT>
__device__ __forceinline__ const void* elem_ptr(const void* p, int64_t i) {
  return static_cast<const typename Elem<DT>::type*>(p) + i;
}
template <int DT>
__device__ __forceinline__ void* elem_ptr(void* p, int64_t i) {
  return static_cast<typename Elem<DT>::type*>(p) + i;
}

template <int DT, int VB, int U>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(const KeepArgs a, int segs) {
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int c;
  if (!place_of(a, segs, U, r, c)) return;
  void* stage = warp_stage<DT, VB>();
  Span<DT, VB> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    x[u].load(elem_ptr<DT>(a.x, r * a.ld_x + c + u * kSpan), a.W - c - u * kSpan);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t w[kRunWords<DT>];
    x[u].runs(stage, w);
    Run8 v;
    run_unpack<DT>(w, v);
    keep_run<DT>(a, r, c + u * kSpan, 1, 0, w, v);
  }
}

template <int DT, int VB, int U>
__global__ void __launch_bounds__(kThreads) restore_kernel(const KeepArgs a, int segs) {
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int c;
  if (!place_of(a, segs, U, r, c)) return;
  void* stage = warp_stage<DT, VB>();
  Kept k[U];
#pragma unroll
  for (int u = 0; u < U; ++u) k[u] = kept_run(a, r, c + u * kSpan, 1, 0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Run8 v;
    e4m3x8_to_float(k[u].codes, block_scale(k[u].byte), v);
    span_store<DT, VB>(elem_ptr<DT>(a.out, r * a.ld_out + c + u * kSpan), a.W - c - u * kSpan,
                       stage, v);
  }
}

// s(g): to fp32's last bits for fp32 rows; by the hardware's exponential and reciprocal
// (2^-21 of the result, results below 2^-126 are 0) where y is rounded to 16 bits.
// Two at a time: a multiplication or addition of two fp32 is one instruction.
template <int DT>
__device__ __forceinline__ f32x2 sigmoid2(f32x2 g) {
  if constexpr (DT == kF32) {
    const float2 f = unpack2(g);
    return pack2(1.0f / (1.0f + expf(-f.x)), 1.0f / (1.0f + expf(-f.y)));
  }
  const float2 k = unpack2(mul2(g, pack2(-kLog2e, -kLog2e)));
  const float2 t = unpack2(add2(pack2(ex2(k.x), ex2(k.y)), pack2(1.0f, 1.0f)));
  float s0, s1;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(t.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(t.y));
  return pack2(s0, s1);
}
// min and max that keep a NaN.
__device__ __forceinline__ float cap(float g, float L) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(g), "f"(L));
  return y;
}
__device__ __forceinline__ float clip(float u, float L) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(cap(u, L)), "f"(-L));
  return y;
}
// h where it is positive (or NaN), else 0.
__device__ __forceinline__ float positive(float h) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(h));
  return y;
}

template <int DT, int VB, int U, int ACT, bool LIMIT>
__global__ void __launch_bounds__(kThreads) act_kernel(const KeepArgs a, int segs) {
  constexpr int kHalves = ACT == kActSwiglu ? 2 : 1;
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int c;
  if (!place_of(a, segs, U, r, c)) return;
  void* stage = warp_stage<DT, VB>();
  Span<DT, VB> x[U][kHalves];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      x[u][h].load(elem_ptr<DT>(a.x, r * a.ld_x + h * a.W + c + u * kSpan), a.W - c - u * kSpan);
  const float L = a.limit;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t w[kHalves][kRunWords<DT>];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) x[u][h].runs(stage, w[h]);
    Run8 g, up, y;
    run_unpack<DT>(w[0], g);
    if constexpr (ACT == kActSwiglu) {
      run_unpack<DT>(w[kHalves - 1], up);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        f32x2 gc = pack2(g.v[i], g.v[i + 1]), uc = pack2(up.v[i], up.v[i + 1]);
        if (LIMIT) {
          gc = pack2(cap(g.v[i], L), cap(g.v[i + 1], L));
          uc = pack2(clip(up.v[i], L), clip(up.v[i + 1], L));
        }
        const float2 f = unpack2(mul2(mul2(gc, sigmoid2<DT>(gc)), uc));
        y.v[i] = f.x;
        y.v[i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = positive(g.v[i]);
        y.v[i] = h * h;
      }
    }
    const int cu = c + u * kSpan;
    span_store<DT, VB>(elem_ptr<DT>(a.out, r * a.ld_out + cu), a.W - cu, stage, y);
    if (!a.codes) continue;
    keep_run<DT>(a, r, cu, kHalves, 0, w[0], g);
    if constexpr (ACT == kActSwiglu) keep_run<DT>(a, r, cu, kHalves, 1, w[kHalves - 1], up);
  }
}

// (16-bit rows: five blocks an SM, 48 registers a thread)
template <int DT, int VB, int U, int ACT, bool LIMIT>
__global__ void __launch_bounds__(kThreads, DT == kF32 ? 1 : 5) act_grad_kernel(const KeepArgs a, int segs) {
  constexpr int kHalves = ACT == kActSwiglu ? 2 : 1;
  pdl_trigger();
  pdl_wait();
  int64_t r;
  int c;
  if (!place_of(a, segs, U, r, c)) return;
  void* stage = warp_stage<DT, VB>();
  Span<DT, VB> x[U];
  Kept k[U][kHalves];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int cu = c + u * kSpan;
    x[u].load(elem_ptr<DT>(a.x, r * a.ld_x + cu), a.W - cu);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) k[u][h] = kept_run(a, r, cu, kHalves, h);
  }
  const float L = a.limit;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int cu = c + u * kSpan;
    uint32_t w[kRunWords<DT>];
    x[u].runs(stage, w);
    Run8 g, up, d;
    run_unpack<DT>(w, d);
    e4m3x8_to_float(k[u][0].codes, block_scale(k[u][0].byte), g);
    if constexpr (ACT == kActSwiglu) {
      e4m3x8_to_float(k[u][kHalves - 1].codes, block_scale(k[u][kHalves - 1].byte), up);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const f32x2 gk = pack2(g.v[i], g.v[i + 1]), uk = pack2(up.v[i], up.v[i + 1]);
        f32x2 gc = gk, uc = uk;
        if (LIMIT) {
          gc = pack2(cap(g.v[i], L), cap(g.v[i + 1], L));
          uc = pack2(clip(up.v[i], L), clip(up.v[i + 1], L));
        }
        const f32x2 dd = pack2(d.v[i], d.v[i + 1]), s = sigmoid2<DT>(gc), gs = mul2(gc, s);
        // s (1 + g (1 - s)) = s + g s (1 - s), times u before dy: dy u may pass fp32's range where
        // the slope is small or 0
        const f32x2 rest = fma2(s, pack2(-1.0f, -1.0f), pack2(1.0f, 1.0f));
        const float2 dg = unpack2(mul2(dd, mul2(uc, fma2(gs, rest, s))));
        const float2 du = unpack2(mul2(dd, gs));
        const float2 gf = unpack2(gk), uf = unpack2(uk);
        g.v[i] = LIMIT && gf.x > L ? 0.0f : dg.x;
        g.v[i + 1] = LIMIT && gf.y > L ? 0.0f : dg.y;
        up.v[i] = LIMIT && fabsf(uf.x) > L ? 0.0f : du.x;
        up.v[i + 1] = LIMIT && fabsf(uf.y) > L ? 0.0f : du.y;
      }
      span_store<DT, VB>(elem_ptr<DT>(a.out, r * a.ld_out + a.W + cu), a.W - cu, stage, up);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g.v[i] = 2.0f * (d.v[i] * positive(g.v[i]));  // 2 dy may overflow
    }
    span_store<DT, VB>(elem_ptr<DT>(a.out, r * a.ld_out + cu), a.W - cu, stage, g);
  }
}

int size_of(int dtype) { return dtype == kF32 ? 4 : 2; }

// Widest access to rows of W values, the second half W values further on.
int width(const void* p, int64_t ld, int W, int dtype) {
  return access_bytes(p, ld * size_of(dtype), (int64_t)W * size_of(dtype));
}

template <typename K>
cudaError_t go(K kernel, const KeepArgs& a, int u, cudaStream_t s) {
  const int segs = (a.W + u * kSpan - 1) / (u * kSpan);
  const int64_t blocks = ((int64_t)a.R * segs + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a, segs);
}

// U spans a warp where that leaves the device enough warps (16 an SM), else one: 128 rows of
// 1024 take 3.2 us with one span a warp.  (Rows of a few spans gain least: 5001 x 1407 of fp32,
// six spans a row, are kept in 7.4 us, by one span a warp in 6.5; of 16 bits both in 6.5.)
constexpr int64_t kManyWarps = 152 * 16;
int spans(const KeepArgs& a, int u) {
  return (int64_t)a.R * ((a.W + u * kSpan - 1) / (u * kSpan)) >= kManyWarps ? u : 1;
}

#define MOE_BY_WIDTH(KERNEL, DT, U, vb, ...)                                                      \
  const bool many = spans(a, U) == U;                                                             \
  switch (vb) {                                                                                   \
    case 16:                                                                                      \
      return many ? go(KERNEL<DT, 16, U __VA_ARGS__>, a, U, s)                                    \
                  : go(KERNEL<DT, 16, 1 __VA_ARGS__>, a, 1, s);                                   \
    case 8:                                                                                       \
      return many ? go(KERNEL<DT, 8, U __VA_ARGS__>, a, U, s)                                     \
                  : go(KERNEL<DT, 8, 1 __VA_ARGS__>, a, 1, s);                                    \
    case 4:                                                                                       \
      return many ? go(KERNEL<DT, 4, U __VA_ARGS__>, a, U, s)                                     \
                  : go(KERNEL<DT, 4, 1 __VA_ARGS__>, a, 1, s);                                    \
    default: break;                                                                               \
  }                                                                                               \
  if constexpr (DT != kF32)                                                                       \
    return many ? go(KERNEL<DT, 2, U __VA_ARGS__>, a, U, s)                                       \
                : go(KERNEL<DT, 2, 1 __VA_ARGS__>, a, 1, s);                                      \
  return cudaErrorInvalidValue;
#define MOE_COMMA ,

template <int DT>
cudaError_t checkpoint_typed(const KeepArgs& a, cudaStream_t s) {
  MOE_BY_WIDTH(checkpoint_kernel, DT, 4, width(a.x, a.ld_x, a.W, DT))
}
// (fp32: two spans 5001 x 1407 6.1 us, 4096 x 7168 30.1; four 6.8 and 30.9)
template <int DT>
cudaError_t restore_typed(const KeepArgs& a, cudaStream_t s) {
  MOE_BY_WIDTH(restore_kernel, DT, (DT == kF32 ? 2 : 4), width(a.out, a.ld_out, a.W, DT))
}
template <int DT, int ACT, bool LIMIT>
cudaError_t act_typed(const KeepArgs& a, cudaStream_t s) {
  const int vb = std::min(width(a.x, a.ld_x, a.W, DT), width(a.out, a.ld_out, a.W, DT));
  MOE_BY_WIDTH(act_kernel, DT, 2, vb, MOE_COMMA ACT MOE_COMMA LIMIT)
}
template <int DT, int ACT, bool LIMIT>
cudaError_t act_grad_typed(const KeepArgs& a, cudaStream_t s) {
  const int vb = std::min(width(a.x, a.ld_x, a.W, DT), width(a.out, a.ld_out, a.W, DT));
  MOE_BY_WIDTH(act_grad_kernel, DT, 2, vb, MOE_COMMA ACT MOE_COMMA LIMIT)
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
namespace {

template <int DT>
cudaError_t act_any(const KeepArgs& a, int act, cudaStream_t s) {
  if (act == kActRelu2) return act_typed<DT, kActRelu2, false>(a, s);
  return a.limit > 0.0f ? act_typed<DT, kActSwiglu, true>(a, s)
                        : act_typed<DT, kActSwiglu, false>(a, s);
}
template <int DT>
cudaError_t act_grad_any(const KeepArgs& a, int act, cudaStream_t s) {
  if (act == kActRelu2) return act_grad_typed<DT, kActRelu2, false>(a, s);
  return a.limit > 0.0f ? act_grad_typed<DT, kActSwiglu, true>(a, s)
                        : act_grad_typed<DT, kActSwiglu, false>(a, s);
}

}  // namespace

cudaError_t launch_expert_act(const KeepArgs& a, int act, int dtype, cudaStream_t s) {
  return dtype == kF32    ? act_any<kF32>(a, act, s)
         : dtype == kBf16 ? act_any<kBf16>(a, act, s)
                          : act_any<kF16>(a, act, s);
}
cudaError_t launch_expert_act_grad(const KeepArgs& a, int act, int dtype, cudaStream_t s) {
  return dtype == kF32    ? act_grad_any<kF32>(a, act, s)
         : dtype == kBf16 ? act_grad_any<kBf16>(a, act, s)
                          : act_grad_any<kF16>(a, act, s);
}

}  // namespace moe
