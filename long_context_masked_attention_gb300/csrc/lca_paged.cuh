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

// Request i with its lengths clamped to what the tensors hold (paged_begin
// reports those that need it).
__device__ __forceinline__ SegInfo paged_seg(const PagedAttnArgs& a, int i) {
  const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
  const int room = a.max_pages * a.page_size;
  SegInfo s{};
  s.q_off = min(max(r0, 0), a.Tq);
  s.q_len = min(max(r1, s.q_off), a.Tq) - s.q_off;
  s.k_len = min(max(kl, 0), room);
  return s;
}

// Key ranges are found once per item, by calls and not inline: short batches
// wait for instructions more than for data, so what is not a tile's work is
// kept small.
static __device__ __noinline__ Span paged_span(const PagedAttnArgs& a, int q_len, int k_len, int i) {
  SegInfo sg{};
  sg.q_len = q_len;
  sg.k_len = k_len;
  return row_span(a.mask, sg, i);
}

// Keys that some of the tokens [i0, i1) of a request attends: in every family
// the bounds of a row's intervals do not decrease from token to token, but
// for the first lower bound, which may fall to 0 at the last rows, and for
// GLOBAL_SLIDING's first rows, whose one interval holds all keys; so the two
// outer rows give the hull.
static __device__ __noinline__ Span hull(const PagedAttnArgs& a, int q_len, int k_len, int i0, int i1) {
  const Span s = paged_span(a, q_len, k_len, i0), t = paged_span(a, q_len, k_len, i1 - 1);
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

// Sums of one row over pieces that hold it unnormalised, by a whole warp:
// piece k has its values (128) at at(k), its maximum at stat(k)[0] and its sum
// of exponentials at stat(k)[gap].  Lane j gets values 4 j .. 4 j + 3.  All
// loads of eight pieces are under way at once: a trip to L2 is what this costs.
template <typename At, typename Stat>
__device__ __forceinline__ void join_row(int n, At at, Stat stat, int gap, float& m, float& l, float (&o)[4]) {
  const int lane = threadIdx.x & 31;
  // lane k: piece k of the first 32
  const float m0 = lane < n ? __ldcg(stat(lane)) : -INFINITY, l0 = lane < n ? __ldcg(stat(lane) + gap) : 0.f;
  m = m0;
  for (int k = lane + 32; k < n; k += 32) m = fmaxf(m, __ldcg(stat(k)));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  l = 0.f;
  o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll 1
  for (int b = 0; b < n; b += 32) {
    float mk = m0, lk = l0;
    if (b > 0) {
      mk = b + lane < n ? __ldcg(stat(b + lane)) : -INFINITY;
      lk = b + lane < n ? __ldcg(stat(b + lane) + gap) : 0.f;
    }
    const float f = lk != 0.f ? ex2_approx(mk - m) : 0.f;
    l = fmaf(f, lk, l);
    const int here = min(32, n - b);
#pragma unroll 1
    for (int k = 0; k < here; k += 8) {
      float4 z[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) z[u] = __ldcg(reinterpret_cast<const float4*>(at(b + min(k + u, here - 1))) + lane);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float fk = __shfl_sync(~0u, f, min(k + u, 31));
        if (k + u < here && fk != 0.f) {  // a piece without keys leaves its values unwritten
          o[0] = fmaf(fk, z[u].x, o[0]);
          o[1] = fmaf(fk, z[u].y, o[1]);
          o[2] = fmaf(fk, z[u].z, o[2]);
          o[3] = fmaf(fk, z[u].w, o[3]);
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
}

// a / b of the line's positions, once in code
static __device__ __noinline__ long long line_div(long long a, long long b) { return a / b; }

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
