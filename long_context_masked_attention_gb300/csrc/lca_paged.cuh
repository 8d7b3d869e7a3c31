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
  // sign bits set where the exponent is all ones (infinities, NaN); the other
  // bits say nothing
  static __device__ __forceinline__ uint32_t not_finite(uint32_t x) { return (x & 0x7FFF7FFFu) + 0x00800080u; }
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
  static __device__ __forceinline__ uint32_t not_finite(uint32_t x) { return (x & 0x7FFF7FFFu) + 0x04000400u; }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
};

// The status word of a call: status[0] the code, status[1] where it was raised,
// set as one 64-bit word.  Lengths and table entries that cannot be used
// (kStatusDeviceArg) are reported and the call goes on with what the header
// promises for them; only a wait that ran out ends it, and replaces such a
// report.  Of two reports of a kind the first stays.
__device__ __forceinline__ void paged_report(int* status, int code, int where) {
  auto* word = reinterpret_cast<unsigned long long*>(status);
  const unsigned long long x = static_cast<unsigned>(code) | static_cast<unsigned long long>(where) << 32;
  const unsigned long long was = atomicCAS(word, 0ull, x);
  if (code == kStatusTimeout && was != 0 && static_cast<int>(was) != kStatusTimeout) atomicCAS(word, was, x);
}
__device__ __forceinline__ bool paged_timed_out(const int* status) {
  return *reinterpret_cast<const volatile int*>(status) == kStatusTimeout;
}

// mbar_wait that gives up when its time is over or another wait's was, and for
// no other report.
__device__ __forceinline__ bool paged_wait(uint64_t* bar, uint32_t parity, int* status, uint64_t limit_ns, int where) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 63u) != 0) continue;
    if (paged_timed_out(status)) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      paged_report(status, kStatusTimeout, where);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// j / page_size for j in [0, 2^30) (see page_divisor), without a division's chain of instructions.
__device__ __forceinline__ int page_index(const PagedAttnArgs& a, int j) {
  return static_cast<int>(__umulhi(static_cast<uint32_t>(j), a.page_mul) >> a.page_shift);
}

__device__ __forceinline__ bool in_span(const Span& s, int j) {
  return (j >= s.a0 && j < s.b0) || (j >= s.a1 && j < s.b1);
}

// Rows and keys of request i, clamped to what the tensors hold
// (paged_begin_kernel reports lengths that need it).
__device__ __forceinline__ SegInfo paged_rows(const PagedAttnArgs& a, int i) {
  const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
  const int room = a.max_pages * a.page_size;
  SegInfo s{};
  s.q_off = min(max(r0, 0), a.Tq);
  s.q_len = min(max(r1, s.q_off), a.Tq) - s.q_off;
  s.k_len = min(max(kl, 0), room);
  return s;
}

// Those of them that attention serves.  Where ctx_len says how many tokens
// came before the rows, the keys end with the last row and the rows with the
// last key, so that the rows are the last of the keys again; the rows behind
// have no key (clear_unowned_rows).
__device__ __forceinline__ SegInfo paged_seg(const PagedAttnArgs& a, int i) {
  SegInfo s = paged_rows(a, i);
  if (a.ctx_len) {
    const int first = min(max(a.ctx_len[i], 0), a.max_pages * a.page_size);
    s.k_len = min(s.k_len, first + s.q_len);
    s.q_len = max(s.k_len - first, 0);
  }
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
__device__ __forceinline__ Span hull_of(const Span& s, const Span& t) {
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

static __device__ __noinline__ Span hull(const PagedAttnArgs& a, int q_len, int k_len, int i0, int i1) {
  const Span s = paged_span(a, q_len, k_len, i0);
  return hull_of(s, i1 - 1 > i0 ? paged_span(a, q_len, k_len, i1 - 1) : s);
}

// Whether the kernel for few rows serves a request with q_len new tokens.
__device__ __forceinline__ bool few_rows(const PagedAttnArgs& a, int q_len) {
  return static_cast<long long>(q_len) * a.G <= a.few;
}

// Sums of R rows over n pieces that hold them unnormalised, by a whole warp:
// piece(k) has kRowsOf x 128 values, the rows' maxima, then their sums of
// exponentials.  Lane j gets values 4 j .. 4 j + 3 of the rows row0 .. row0 +
// R - 1, and the maximum and sum of row row0 + j / (32 / R).  The loads of P
// pieces of all rows are under way at once: a trip to L2 is what this costs.
template <int kRowsOf, int R, int P, typename Piece>
__device__ __forceinline__ void join_rows(int n, Piece piece, int row0, float& m, float& l, float (&o)[R][4]) {
  constexpr int W = 32 / R;  // pieces whose factors are in lanes at once
  const int lane = threadIdx.x & 31, p = lane % W, stat = kRowsOf * kHeadDim + row0 + lane / W;
  const float m0 = p < n ? __ldcg(piece(p) + stat) : -INFINITY;
  const float l0 = p < n ? __ldcg(piece(p) + stat + kRowsOf) : 0.f;
  float4 z[P][R];
  auto load = [&](int k) {
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const float* y = piece(min(k + u, n - 1)) + row0 * kHeadDim;
#pragma unroll
      for (int r = 0; r < R; ++r) z[u][r] = __ldcg(reinterpret_cast<const float4*>(y + r * kHeadDim) + lane);
    }
  };
  load(0);
  m = m0;
  for (int k = p + W; k < n; k += W) m = fmaxf(m, __ldcg(piece(k) + stat));
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  l = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
#pragma unroll 1
  for (int b = 0; b < n; b += W) {
    float mk = m0, lk = l0;
    if (b > 0) {
      mk = b + p < n ? __ldcg(piece(b + p) + stat) : -INFINITY;
      lk = b + p < n ? __ldcg(piece(b + p) + stat + kRowsOf) : 0.f;
    }
    // a piece without keys leaves its values unwritten: -1 marks it.  A factor
    // that has become 0 is still used, for values that are not finite
    const float f = lk != 0.f ? ex2_approx(mk - m) : -1.f;
    l = fmaf(f, lk, l);
    const int here = min(W, n - b);
#pragma unroll 1
    for (int k = 0; k < here; k += P) {
      if (b + k > 0) load(b + k);
#pragma unroll
      for (int u = 0; u < P; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float fk = __shfl_sync(~0u, f, r * W + min(k + u, W - 1));
          if (k + u < here && !(fk < 0.f)) {
            o[r][0] = fmaf(fk, z[u][r].x, o[r][0]);
            o[r][1] = fmaf(fk, z[u][r].y, o[r][1]);
            o[r][2] = fmaf(fk, z[u][r].z, o[r][2]);
            o[r][3] = fmaf(fk, z[u][r].w, o[r][3]);
          }
        }
    }
  }
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
}

// a / b of the line's positions (not negative), once in code; 32 bits are
// enough for most calls and a fraction of the work
static __device__ __noinline__ long long line_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
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
