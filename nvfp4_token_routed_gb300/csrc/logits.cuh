// logits.cuh -- reading and writing logits of the three types, and the softmax
// pieces that the objectives share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "loss.h"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Two fp32 values in one 64-bit register, multiplied and added by one instruction.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 pack2(float2 v) { return pack2(v.x, v.y); }
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 16 bytes of logits: 4 fp32 or 8 16-bit values, handled in pairs.
template <int DT>
struct Vec {
  static constexpr int kElems = DT == kF32 ? 4 : 8;
  static constexpr int kPairs = kElems / 2;
  // The bits of -inf, four bytes of them.
  static constexpr uint32_t kNegInf = DT == kF32 ? 0xFF800000u : DT == kBf16 ? 0xFF80FF80u
                                                                            : 0xFC00FC00u;
  uint4 v;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
  __device__ __forceinline__ void set_word(int i, uint32_t w) {
    (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = w;
  }
  __device__ __forceinline__ void fill(uint32_t w) { v = make_uint4(w, w, w, w); }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (DT == kF32)
      return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    const uint32_t w = word(i);
    if constexpr (DT == kBf16)
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ __forceinline__ void set_pair(int i, float2 f) {
    if constexpr (DT == kF32) {
      set_word(2 * i, __float_as_uint(f.x));
      set_word(2 * i + 1, __float_as_uint(f.y));
    } else if constexpr (DT == kBf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      set_word(i, *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      set_word(i, *reinterpret_cast<const uint32_t*>(&h));
    }
  }
  // Words of elementwise maxima (a NaN gives way to the other operand).
  static __device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
    if constexpr (DT == kF32)
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    uint32_t r;
    if constexpr (DT == kBf16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    if constexpr (DT == kF16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float max_of_word(uint32_t w) {
    if constexpr (DT == kF32) return __uint_as_float(w);
    if constexpr (DT == kBf16)
      return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return fmaxf(f.x, f.y);
  }
};

// A softmax's running pair: a reference logit m and s = sum 2^(z c - k), where k is m c
// rounded: one fused multiply-add gives each exponent with a single rounding, and
// rescaling from one reference to another by 2^(k - k') takes k as it is.  The reference is
// the largest logit of the first ones seen; larger ones move it only when their exponent
// passes kMaxExponent (s stays far inside fp32), so that the exponentials need not wait
// for the maximum.  What rounding takes from k stays in the exponents of the reference
// itself: half a unit in the last place, so 64 at most for |k| < kNearRef, which the sums'
// range holds, but more than fp32's soon after, where finite masks (-1e10, -1e30, the type's
// lowest value) may be the only logits of a set.  From kNearRef on the exponents are
// (z - m) c.  Distinct logits on either side of it are 128 or more apart in their exponents,
// so sums of the two kinds never weigh in one another.  A set without a finite logit has
// m = -inf, s = 0; a NaN or +inf logit makes s NaN.
constexpr float kNearRef = 2147483648.0f;  // 2^31
constexpr float kMaxExponent = 24.0f;
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float ref_exponent(float m, float c) { return __fmul_rn(m, c); }
__device__ __forceinline__ bool near_ref(float k) { return fabsf(k) < kNearRef; }
// Exponent of logit z over the finite reference m.
__device__ __forceinline__ float exponent(float z, float m, float c) {
  const float k = ref_exponent(m, c);
  return near_ref(k) ? fmaf(z, c, -k) : (z - m) * c;
}
// Natural logarithm of logit z's weight over the finite reference m.  A token of the type's
// lowest value keeps a finite one of about that size: its exponent, 1.44 times as large,
// may pass fp32 where the logarithm does not.
__device__ __forceinline__ float log_weight(float z, float m, float c, float inv_tau) {
  const float e = exponent(z, m, c);
  return isinf(e) ? (z - m) * inv_tau : e * kLn2;
}
// One logit as a pair.
__device__ __forceinline__ MaxSum one_logit(float z, float c) {
  return {z, z == -INFINITY ? 0.0f : ex2(exponent(z, z, c))};
}
// Exponent that takes sums over reference m to the finite reference `to`.
__device__ __forceinline__ float rescale(float m, float to, float c) {
  const float k = ref_exponent(to, c);
  return near_ref(k) ? __fsub_rn(ref_exponent(m, c), k) : (m - to) * c;
}
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m), r = finite_ref(m);
  return {m, a.s * ex2(rescale(a.m, r, c)) + b.s * ex2(rescale(b.m, r, c))};
}
// Pairs of lanes 0..n-1 merged in every lane, n a power of two; the order of the
// additions does not depend on the lane.
__device__ __forceinline__ MaxSum warp_merge(MaxSum v, float c, int n) {
  float m = v.m;
  for (int off = n / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  float s = v.s * ex2(rescale(v.m, finite_ref(m), c));
  for (int off = n / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  return {m, s};
}
// Sum of 2^((z - m) c) over a vector, for references that are not near (rare: not inlined).
template <int DT>
__device__ __noinline__ float far_sum(uint4 v, float m, float c) {
  const Vec<DT> d = {v};
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < Vec<DT>::kPairs; ++j) {
    const float2 x = d.pair(j);
    s += ex2((x.x - m) * c) + ex2((x.y - m) * c);
  }
  return s;
}
// The vectors d added to a pair.
template <int DT, int U>
__device__ __forceinline__ MaxSum add_vecs(MaxSum v, const Vec<DT> (&d)[U], float c) {
  uint32_t w = d[0].v.x;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = u == 0 ? 1 : 0; j < 4; ++j) w = Vec<DT>::max_word(w, d[u].word(j));
  const float top = Vec<DT>::max_of_word(w);
  if (v.m == -INFINITY) v.m = top;
  while (true) {
    const float r = finite_ref(v.m), k = ref_exponent(r, c);
    f32x2 acc[2] = {0, 0};
    if (near_ref(k)) {
      const f32x2 c2 = pack2(c, c), neg = pack2(-k, -k);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < Vec<DT>::kPairs; ++j) {
          const float2 x = unpack2(fma2(pack2(d[u].pair(j)), c2, neg));
          acc[j & 1] = add2(acc[j & 1], pack2(ex2(x.x), ex2(x.y)));
        }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        acc[0] = add2(acc[0], pack2(far_sum<DT>(d[u].v, r, c), 0.0f));
    }
    if (top > r && exponent(top, r, c) > kMaxExponent) {  // not with r = top: ends
      v.s *= ex2(rescale(v.m, top, c));
      v.m = top;
      continue;
    }
    const float2 s = unpack2(add2(acc[0], acc[1]));
    return {v.m, v.s + (s.x + s.y)};
  }
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
