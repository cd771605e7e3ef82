// logits.cuh -- reading and writing logits of the three types, and the softmax
// pieces that the objectives share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "loss.h"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;

template <int DT>
__device__ __forceinline__ float load_logit(const typename LogitType<DT>::type* p) {
  if constexpr (DT == kF32) return *p;
  if constexpr (DT == kBf16) return __uint_as_float((uint32_t)*p << 16);
  if constexpr (DT == kF16) return __half2float(__ushort_as_half(*p));
}
template <int DT>
__device__ __forceinline__ void store_logit(typename LogitType<DT>::type* p, float v) {
  if constexpr (DT == kF32) *p = v;
  if constexpr (DT == kBf16) *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  if constexpr (DT == kF16) *p = __half_as_ushort(__float2half_rn(v));
}

// 2^x by the hardware instruction (2 ulp; results below 2^-126 become 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A softmax's running pair: the largest logit m and s = sum 2^((z - m) c).
// Scaling by the distance to m before exponentiating keeps every term in [0, 1]
// for any finite logits; a set without a finite logit has m = -inf, s = 0; a
// NaN or +inf logit makes s NaN.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float r = finite_ref(m);
  return {m, a.s * ex2((a.m - r) * c) + b.s * ex2((b.m - r) * c)};
}
__device__ __forceinline__ MaxSum warp_merge(MaxSum v, float c) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const MaxSum o = {__shfl_xor_sync(0xFFFFFFFFu, v.m, off),
                      __shfl_xor_sync(0xFFFFFFFFu, v.s, off)};
    v = merge(v, o, c);
  }
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

// Index i of an int32 or int64 array; a value outside the int32 range reads as -1.
__device__ __forceinline__ int load_id(const void* ids, int ids64, int64_t i) {
  if (!ids64) return static_cast<const int32_t*>(ids)[i];
  const long long v = static_cast<const long long*>(ids)[i];
  return v < 0 || v > INT32_MAX ? -1 : (int)v;
}

}  // namespace moe
