// lca_paged.cuh — device code shared by the kernels of attention over a paged
// cache: 16-bit pairs of either type, requests, key ranges, sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lca_paged.h"
#include "sm103.cuh"

namespace lca {

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ bool not_finite(uint32_t x) {
    return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
};
template <>
struct Half2<__half> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ bool not_finite(uint32_t x) {
    return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
};

__device__ __forceinline__ bool in_span(const Span& s, int j) {
  return (j >= s.a0 && j < s.b0) || (j >= s.a1 && j < s.b1);
}

// Request i with its lengths clamped to what the tensors hold; `flag` reports
// those that needed it.
__device__ __forceinline__ SegInfo paged_seg(const PagedAttnArgs& a, int i, bool flag) {
  const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
  const int room = a.max_pages * a.page_size;
  if (flag && (r0 < 0 || r1 < r0 || r1 > a.Tq || kl < 0 || kl > room)) raise_status(a.status, kStatusDeviceArg, 50);
  SegInfo s{};
  s.q_off = min(max(r0, 0), a.Tq);
  s.q_len = min(max(r1, s.q_off), a.Tq) - s.q_off;
  s.k_len = min(max(kl, 0), room);
  return s;
}

// Keys that some of the tokens [i0, i1) of a request attends: in every family
// the bounds of a row's intervals do not decrease from token to token, but
// for the first lower bound, which may fall to 0 at the last rows, and for
// GLOBAL_SLIDING's first rows, whose one interval holds all keys; so the two
// outer rows give the hull.
__device__ __forceinline__ Span hull(const MaskCtx& m, const SegInfo& sg, int i0, int i1) {
  const Span s = row_span(m, sg, i0), t = row_span(m, sg, i1 - 1);
  Span h;
  h.a0 = min(s.a0, t.a0);
  h.b0 = max(max(s.b0, t.b0), h.a0);
  h.a1 = h.b1 = h.b0;
  if (t.a1 < t.b1) {
    h.a1 = s.a1 < s.b1 ? min(s.a1, t.a1) : t.a1;
    h.b1 = max(t.b1, h.b0);
    if (h.a1 <= h.b0) {  // they touch
      h.b0 = h.b1;
      h.a1 = h.b1;
    }
  }
  return h;
}

// Whether the kernel for few rows serves a request with q_len new tokens.
__device__ __forceinline__ bool few_rows(const PagedAttnArgs& a, int q_len) {
  return static_cast<long long>(q_len) * a.G <= a.few;
}

// Inclusive sum over a block of 1024 threads; `total` gets the whole sum.
// part: shared memory, free again when the call returns on every thread.
__device__ __forceinline__ long long block_scan(long long x, long long (&part)[32], long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  long long w = part[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(~0u, w, 31);
  const long long before = __shfl_sync(~0u, w, (warp + 31) & 31);
  __syncthreads();
  return warp > 0 ? x + before : x;
}

}  // namespace lca
