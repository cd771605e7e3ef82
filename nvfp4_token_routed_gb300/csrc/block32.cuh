// block32.cuh -- blocks of 32 values that share a power of two: exponents, and the
// reading and writing of runs of 8 values of any alignment.
//
// A block holds x_i = 2^e q_i with q_i of an 8- or 4-bit float type whose largest value
// is qmax.  e is the smallest exponent with max |x_i| <= qmax 2^e, so that no value is
// cut off and each is off by at most half a step of its type (or of its smallest step).
// With max |x_i| = m 2^k, 1 <= m < 2, and qmax = f 2^j: e = k - j + (m > f), which needs
// the bits of the largest magnitude and no division.  e is kept in [-127, 127] as the
// byte e + 127; byte 255 marks a block with an infinity or a NaN, which reads as NaN.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "logits.cuh"
#include "loss.h"
#include "ptx.cuh"

namespace moe {

struct E4m3 {  // qmax = 448 = 1.75 * 2^8
  static constexpr int kMaxExp = 8;
  static constexpr uint32_t kMaxMantissa = 0x600000u;
};
struct E2m1 {  // qmax = 6 = 1.5 * 2^2
  static constexpr int kMaxExp = 2;
  static constexpr uint32_t kMaxMantissa = 0x400000u;
};

// Scale byte of a block from the bits of its largest magnitude.
template <typename F>
__device__ __forceinline__ uint32_t block_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int b = (int)(amax_bits >> 23) - F::kMaxExp + ((amax_bits & 0x7FFFFFu) > F::kMaxMantissa);
  return (uint32_t)max(b, 0);  // fp32 subnormals come out below 0 as well
}
// 2^-e, for byte 255 0: its codes are zeros.
__device__ __forceinline__ float block_inverse(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^e, NaN for byte 255.
__device__ __forceinline__ float block_scale(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// 8 values of a row in fp32.
struct Run8 {
  float v[8];
};

template <int DT>
struct Elem {
  using type = uint16_t;
};
template <>
struct Elem<kF32> {
  using type = uint32_t;
};
template <int DT>
__device__ __forceinline__ float elem_to_float(uint32_t b) {
  if constexpr (DT == kF32) return __uint_as_float(b);
  if constexpr (DT == kBf16) return __uint_as_float(b << 16);
  if constexpr (DT == kF16) return __half2float(__ushort_as_half((unsigned short)b));
}
template <int DT>
__device__ __forceinline__ uint32_t float_to_elem(float v) {
  if constexpr (DT == kF32) return __float_as_uint(v);
  if constexpr (DT == kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  if constexpr (DT == kF16) return __half_as_ushort(__float2half_rn(v));
}

// 32-bit words of 8 elements.
template <int DT>
constexpr int kRunWords = DT == kF32 ? 8 : 4;

// A span: 256 consecutive elements of a row by one warp, run l (elements 8l ... 8l + 7) in
// lane l.  With rows on 16 bytes (VB = 16) a lane reads and writes its run; else accesses of
// VB bytes go by consecutive lanes (a run a lane, its accesses would lie 16 bytes apart and
// each touch 16 sectors) and the runs are put together in shared memory, kSpanBytes a warp.
// n: elements of the row from the span's first on (any number; those past n read as zero and
// are not written).  All lanes take part.
constexpr int kSpan = 256;
template <int DT, int VB>
constexpr int kSpanBytes = VB == 16 ? 16 : kSpan * (DT == kF32 ? 4 : 2);  // 16: not used

template <int DT, int VB>
struct NarrowType {
  using type = uint16_t;
};
template <int DT>
struct NarrowType<DT, 4> {
  using type = uint32_t;
};
template <int DT>
struct NarrowType<DT, 8> {
  using type = uint2;
};

// A span as it was read, and the runs made of it: several spans are read before the first is
// put together.
template <int DT, int VB>
struct Span {
  using V = typename NarrowType<DT, VB>::type;
  static constexpr int kPer = VB / (DT == kF32 ? 4 : 2), kN = kSpan / kPer / 32;
  V t[kN];
  __device__ __forceinline__ void load(const void* p, int n) {
    const int lane = threadIdx.x & 31;
    const V* c = reinterpret_cast<const V*>(p);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      t[i] = V{};
      if ((32 * i + lane) * kPer < n) t[i] = c[32 * i + lane];
    }
  }
  __device__ __forceinline__ void runs(void* stage, uint32_t (&w)[kRunWords<DT>]) const {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // an earlier use of the stage is over
#pragma unroll
    for (int i = 0; i < kN; ++i) reinterpret_cast<V*>(stage)[32 * i + lane] = t[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRunWords<DT> / 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(stage)[lane * (kRunWords<DT> / 4) + i];
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  }
};
template <int DT>
struct Span<DT, 16> {
  uint32_t t[kRunWords<DT>];
  __device__ __forceinline__ void load(const void* p, int n) {
    constexpr int kPer = 16 / (DT == kF32 ? 4 : 2);
    const int lane = threadIdx.x & 31;
    const uint4* c = reinterpret_cast<const uint4*>(p) + lane * (8 / kPer);
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const uint4 q = lane * 8 + i * kPer < n ? c[i] : make_uint4(0u, 0u, 0u, 0u);
      t[4 * i] = q.x, t[4 * i + 1] = q.y, t[4 * i + 2] = q.z, t[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void runs(void*, uint32_t (&w)[kRunWords<DT>]) const {
#pragma unroll
    for (int i = 0; i < kRunWords<DT>; ++i) w[i] = t[i];
  }
};
template <int DT>
__device__ __forceinline__ void run_unpack(const uint32_t (&w)[kRunWords<DT>], Run8& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == kF32)
      r.v[i] = __uint_as_float(w[i]);
    else
      r.v[i] = elem_to_float<DT>((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
  }
}
template <int DT, int VB>
__device__ __forceinline__ void span_store(void* p, int n, void* stage, const Run8& r) {
  constexpr int kSize = DT == kF32 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  uint32_t w[kRunWords<DT>];
#pragma unroll
  for (int i = 0; i < kRunWords<DT>; ++i)
    w[i] = DT == kF32 ? float_to_elem<DT>(r.v[i])
                      : float_to_elem<DT>(r.v[(2 * i) & 7]) |
                            (float_to_elem<DT>(r.v[(2 * i + 1) & 7]) << 16);
  if constexpr (VB == 16) {
    constexpr int kPer = 16 / kSize;
    uint4* c = reinterpret_cast<uint4*>(p) + lane * (8 / kPer);
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i)
      if (lane * 8 + i * kPer < n)
        c[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
    using V = typename NarrowType<DT, VB>::type;
    constexpr int kPer = VB / kSize, kN = kSpan / kPer / 32;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRunWords<DT> / 4; ++i)
      reinterpret_cast<uint4*>(stage)[lane * (kRunWords<DT> / 4) + i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
    V* c = reinterpret_cast<V*>(p);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if ((32 * i + lane) * kPer < n) c[32 * i + lane] = reinterpret_cast<const V*>(stage)[32 * i + lane];
  }
}

// Largest of two magnitudes' bits in each half of a word, one instruction.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Bits (of fp32) of the largest magnitude of a block of 32 values, from the words of the four
// lanes' runs; infinities and NaN come out above every finite value.  16-bit types compare as
// unsigned halves, two at a time; all lanes take part.
template <int DT>
__device__ __forceinline__ uint32_t block_amax(const uint32_t (&w)[kRunWords<DT>]) {
  uint32_t m;
  if constexpr (DT == kF32) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  } else {
    m = max16x2(max16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                max16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    m = max16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(elem_to_float<DT>(m));
  }
}

__device__ __forceinline__ Run8 scaled(const Run8& r, float f) {
  Run8 o;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 t = unpack2(mul2(pack2(r.v[i], r.v[i + 1]), pack2(f, f)));
    o.v[i] = t.x;
    o.v[i + 1] = t.y;
  }
  return o;
}

// E4M3 codes of 8 values times `inv` (|v inv| <= 448), value i in byte i.
__device__ __forceinline__ uint2 e4m3x8(const Run8& r, float inv) {
  uint32_t h[2];
  const Run8 v = scaled(r, inv);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}"
        : "=r"(h[i])
        : "f"(v.v[4 * i]), "f"(v.v[4 * i + 1]), "f"(v.v[4 * i + 2]), "f"(v.v[4 * i + 3]));
  return make_uint2(h[0], h[1]);
}
__device__ __forceinline__ void e4m3x8_to_float(const uint2& c, float scale, Run8& r) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
        " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(w[i]));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = unpack2(mul2(pack2(__half22float2(*reinterpret_cast<__half2*>(&h[j]))),
                                    pack2(scale, scale)));
      r.v[4 * i + 2 * j] = f.x;
      r.v[4 * i + 2 * j + 1] = f.y;
    }
  }
}
// E2M1 codes of 8 values times `inv`, value i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8(const Run8& r, float inv) {
  uint32_t o;
  const Run8 v = scaled(r, inv);
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(o)
      : "f"(v.v[0]), "f"(v.v[1]), "f"(v.v[2]), "f"(v.v[3]), "f"(v.v[4]), "f"(v.v[5]), "f"(v.v[6]),
        "f"(v.v[7]));
  return o;
}
__device__ __forceinline__ void e2m1x8_to_float(uint32_t c, float scale, Run8& r) {
  uint32_t h[4];
  asm("{\n .reg .b8 t0, t1, t2, t3;\n mov.b32 {t0, t1, t2, t3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, t0;\n cvt.rn.f16x2.e2m1x2 %1, t1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, t2;\n cvt.rn.f16x2.e2m1x2 %3, t3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    r.v[2 * i] = f.x * scale;
    r.v[2 * i + 1] = f.y * scale;
  }
}

// Widest access (bytes, at most 16) by which rows of `row_bytes` at base, stride
// ld_bytes, can be read and written.
inline int access_bytes(const void* base, int64_t ld_bytes, int64_t row_bytes) {
  const uint64_t m = reinterpret_cast<uintptr_t>(base) | (uint64_t)ld_bytes | (uint64_t)row_bytes;
  return m % 16 == 0 ? 16 : m % 8 == 0 ? 8 : m % 4 == 0 ? 4 : 2;
}

}  // namespace moe
