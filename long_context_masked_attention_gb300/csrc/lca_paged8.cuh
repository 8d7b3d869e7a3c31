// lca_paged8.cuh — device code of the 8-bit paged cache: e4m3 values and the
// rows' factors.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lca_paged.cuh"
#include "lca_paged8.h"

namespace lca {

// 2^e, e in [-126, 127]
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The exponent of a row's factor as its byte says it.
__device__ __forceinline__ int factor_of(uint32_t byte) {
  return min(max(static_cast<int>(byte) - kScaleBias, kScaleMin), kScaleMax);
}

// Two e4m3 values (the low 16 bits) as fp16 ones, which hold them exactly; NaN stays.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(x));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// 8 bytes, of which those past `bytes` (0 or 8) are zero
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}

// The top bits of the bytes that are NaN.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Two 32-bit values as e4m3 (lo in the low byte); what lies past 448 becomes 448, NaN stays.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 p;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 p, %2, %1;\n\t"
      "cvt.u32.u16 %0, p;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Two fp16 values as e4m3, likewise.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 p;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, %1;\n\t"
      "cvt.u32.u16 %0, p;\n\t}"
      : "=r"(r)
      : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four e4m3 values times 2^e as two pairs of T.  In bf16 the product is exact;
// in fp16 it is rounded and ends at the type's largest.
template <typename T>
struct Dequant;
template <>
struct Dequant<__nv_bfloat16> {
  static __device__ __forceinline__ uint2 quad(uint32_t x, float f) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(x)), b = f16x2_to_float2(e4m3x2_hi_to_f16x2(x));
    return make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(b.x * f, b.y * f));
  }
};
template <>
struct Dequant<__half> {
  static __device__ __forceinline__ float bound(float x) {  // NaN stays
    return x > 65504.f ? 65504.f : x < -65504.f ? -65504.f : x;
  }
  static __device__ __forceinline__ uint2 quad(uint32_t x, float f) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(x)), b = f16x2_to_float2(e4m3x2_hi_to_f16x2(x));
    return make_uint2(Half2<__half>::pack(bound(a.x * f), bound(a.y * f)), Half2<__half>::pack(bound(b.x * f), bound(b.y * f)));
  }
};

}  // namespace lca
