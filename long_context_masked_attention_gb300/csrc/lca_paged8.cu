// lca_paged8.cu — kernels of the 8-bit paged cache: quantising new keys and
// values into their pages, reading pages back, and attention of few rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lca_paged.cuh"
#include "lca_paged8.cuh"
#include "lca_paged_few.cuh"
#include "sm103.cuh"

namespace lca {
namespace {

// ------------------------------------------------------------------ write
// 16 threads per (row, head), for K and V together, as in the 16-bit write:
// each reads 16 bytes of both, the half-warp finds the two rows' largest
// magnitudes (as integers: a positive float's bits are in its order), and each
// thread writes 8 bytes of both.  The factor is a power of two, so dividing by
// it is an exact product and the only rounding is e4m3's.  Reads 512 bytes a
// row and head and writes 258, which bounds it.
template <typename T>
struct Magnitude;
template <>
struct Magnitude<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7F807F80u;
  static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m << 16); }
};
template <>
struct Magnitude<__half> {
  static constexpr uint32_t kInf = 0x7C007C00u;
  static __device__ __forceinline__ float value(uint32_t m) { return __half2float(__ushort_as_half(static_cast<unsigned short>(m))); }
};

// Largest finite magnitude of eight values, as the type's bits.
template <typename T>
__device__ __forceinline__ uint32_t largest(const uint4& x) {
  uint32_t m = 0;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    m = __vmaxu2(m, a & __vcmpltu2(a, Magnitude<T>::kInf));
  }
  return max(m & 0xFFFFu, m >> 16);
}

// The smallest e with 2^e 448 >= m, as far as factors go: 448 = 1.75 2^8.
__device__ __forceinline__ int row_factor(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleMin), kScaleMax);
}

template <typename T>
__device__ __forceinline__ uint2 quantise(const uint4& x, float f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Half2<T>::unpack(w[i]);
    // an infinity would end at 448: it is NaN, so that it is not lost
    const float nan = __uint_as_float(0x7FC00000u);
    r[i] = to_e4m3x2(fabsf(v.x) == INFINITY ? nan : v.x * f, fabsf(v.y) == INFINITY ? nan : v.y * f);
  }
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}

template <typename T>
__global__ void __launch_bounds__(256) paged_write8_kernel(const PagedWrite8Args a) {
  const long long n = static_cast<long long>(a.n_rows) * a.Hkv * 16;  // a multiple of 16: half-warps stay together
  const int piece = threadIdx.x & 15;
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  for (long long t = blockIdx.x * 256LL + threadIdx.x; t < n; t += gridDim.x * 256LL) {
    const long long rh = t >> 4;
    const int head = static_cast<int>(rh % a.Hkv);
    const long long row = rh / a.Hkv;
    const int slot = __ldg(a.slots + row);
    if (slot < 0 || slot >= a.n_slots) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(a.k + row * a.k_stride + head * kHeadDim + piece * 8);
    const uint4 y = *reinterpret_cast<const uint4*>(a.v + row * a.v_stride + head * kHeadDim + piece * 8);
    uint32_t m = largest<T>(x) | largest<T>(y) << 16;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(half, m, d));
    const int ek = row_factor(Magnitude<T>::value(m & 0xFFFFu)), ev = row_factor(Magnitude<T>::value(m >> 16));
    const int page = slot / a.page_size, token = slot % a.page_size;
    const long long at = page * a.page_stride + token * a.token_stride + head * a.head_stride + piece * 8;
    *reinterpret_cast<uint2*>(a.kc + at) = quantise<T>(x, two_to(-ek));
    *reinterpret_cast<uint2*>(a.vc + at) = quantise<T>(y, two_to(-ev));
    if (piece < 2)
      (piece ? a.vs : a.ks)[page * a.scale_page_stride + head * a.scale_head_stride + token] =
          static_cast<uint8_t>((piece ? ev : ek) + kScaleBias);
  }
}

// ------------------------------------------------------------------ read back
// 8 threads per row of K and V, 16 bytes of each read and 32 written, rows in
// the order in which they lie in the cache.
template <typename T>
__global__ void __launch_bounds__(256) paged_read8_kernel(const PagedRead8Args a) {
  const long long n = static_cast<long long>(a.n) * a.page_size * a.Hkv * 8;
  for (long long t = blockIdx.x * 256LL + threadIdx.x; t < n; t += gridDim.x * 256LL) {
    const int piece = static_cast<int>(t & 7);
    const long long r = t >> 3;
    const unsigned inner = a.token_first ? a.page_size : a.Hkv, outer = a.token_first ? a.Hkv : a.page_size;
    const long long ro = r / inner;
    const unsigned in = static_cast<unsigned>(r - ro * inner);
    const long long i = ro / outer;
    const unsigned out = static_cast<unsigned>(ro - i * outer);
    const int token = a.token_first ? in : out, head = a.token_first ? out : in;
    const int page = __ldg(a.pages + i);
    if (page < 0 || page >= a.n_pages) continue;
    const long long at = page * a.page_stride + token * a.token_stride + head * a.head_stride + piece * 16;
    const long long st = page * a.scale_page_stride + head * a.scale_head_stride + token;
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.kc + at)), y = __ldg(reinterpret_cast<const uint4*>(a.vc + at));
    const float fk = two_to(factor_of(__ldg(a.ks + st))), fv = two_to(factor_of(__ldg(a.vs + st)));
    const long long to = i * a.out_page_stride + token * a.out_token_stride + head * a.out_head_stride + piece * 16;
    auto put = [](uint16_t* dst, const uint4& w, float f) {
      const uint2 p = Dequant<T>::quad(w.x, f), q = Dequant<T>::quad(w.y, f), r = Dequant<T>::quad(w.z, f), s = Dequant<T>::quad(w.w, f);
      *reinterpret_cast<uint4*>(dst) = make_uint4(p.x, p.y, q.x, q.y);
      *reinterpret_cast<uint4*>(dst + 8) = make_uint4(r.x, r.y, s.x, s.y);
    };
    put(a.k + to, x, fk);
    put(a.v + to, y, fv);
  }
}

// ------------------------------------------------------------------ attention, few rows
// A warp's share of the line in lca_paged_few.cuh: a key costs 258 bytes.
//
// Mathematics.  With factors 2^ek and 2^ev of a key's rows and e4m3 values k8
// and v8, s = scale 2^ek q.k8 and o = sum e^s 2^ev v8 / sum e^s.  The maximum
// that the sums are kept relative to is that of t = s log2(e) + ev, so the
// weights w = 2^(t - max) of the product with v8 are at most 1 whatever the
// factors, and the sum of exponentials gets w 2^-ev.
//
// Both products take fp16 operands, which hold e4m3 exactly.  q is scaled by a power
// of two per row, so that its largest value is near 2^14: a bf16 q below 2^-28
// of its row's largest loses bits, which shows in scores at 2^-38 of the largest
// product.  w is rounded to fp16 times up to 2^12: keys down to 2^-36 of the
// largest count, below 2^-26 with fewer bits.  The sums go by m = max - 12,
// rounded up: where 12 is less than the last place of a huge score, w stays at
// most 2^12.
//
// A lane's operands come from shared memory by 16-byte loads and are converted
// in registers.  The order of the 128 products of a score, and of the columns of O,
// is free, so a lane takes the bytes that lie together: of key lane / 4 the
// pieces lane % 4 and lane % 4 + 4 (four values are the two registers of one
// k16 step, q permuted to fit), and of the four keys of its rows of V the
// piece lane / 4, whose 16 columns are those of the 16 n8 tiles.  Pieces are
// swizzled so that neither pattern has bank conflicts.
constexpr int kStages8 = 3;
constexpr int kSlice8 = kSlice * 128;                 // of K or V
constexpr int kStage8 = 2 * kSlice8 + 2 * kSlice;     // with the factors' bytes
constexpr int kWarp8 = kStages8 * kStage8;
constexpr int kFewSmem8 = kDecWarps * kWarp8;
static_assert(kWarp8 >= 16 * 132 * 4 && kStage8 % 16 == 0, "the ring holds a warp's sums at the end");

__device__ __forceinline__ uint32_t swizzle8(int key) { return (key & 6) ^ ((key & 1) << 2); }

// 8 bytes, of which those past `bytes` (0 or 8) are zero
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// Values of the q's row for the k16 steps, fp16 of q times 2^-e; returns e.
template <typename T>
__device__ __forceinline__ int load_q(const T* row, int c, uint32_t (&lo)[8], uint32_t (&hi)[8]) {
  uint4 x[4];  // pieces c and c + 4, 16 values each
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(row + 16 * (c + 4 * (i >> 1)) + 8 * (i & 1)));
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = Half2<T>::unpack(word(x[i], k));
      m = fmaxf(m, fabsf(v.x) < INFINITY ? fabsf(v.x) : 0.f);  // a NaN counts as 0 too
      m = fmaxf(m, fabsf(v.y) < INFINITY ? fabsf(v.y) : 0.f);
    }
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
  // the largest lands in [2^14, 2^15), in steps that a float can take: 2^-e
  // itself may be past its range
  const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 1) - 127 - 14;
  const float f0 = two_to(-e / 2), f1 = two_to(-e - -e / 2);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = Half2<T>::unpack(word(x[i], k));
      const uint32_t h = Half2<__half>::pack(v.x * f0 * f1, v.y * f0 * f1);
      const int step = 2 * i + (k >> 1);  // four values a step
      if (k & 1) hi[step] = h; else lo[step] = h;
    }
  return e;
}

template <typename T>
struct Worker8 {
  using Out = T;
  static constexpr int kWarpBytes = kWarp8;
  static constexpr float kBias = 0.f;
  static __device__ __forceinline__ void run(const PagedAttnArgs& a, uint8_t* ring_, int seq, const Request& sg,
                                             const Units& un, int tile, int head, int u0, int n, float* m_out, float* l_out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(ring_);
    const int rows = min(static_cast<int>(min(static_cast<long long>(sg.q_len) * a.G - static_cast<long long>(tile) * kRows, 16LL)), kRows);
    const int r_first = tile * kRows, r_last = r_first + rows - 1;
    const int ra = min(r_first + g, r_last), rb = min(r_first + g + 8, r_last);
    const Span own = paged_span(a, sg.q_len, sg.k_len, min(r_first + (lane & 15), r_last) / a.G);
    auto row_of = [&](int r) {
      return Span{__shfl_sync(~0u, own.a0, r), __shfl_sync(~0u, own.b0, r), __shfl_sync(~0u, own.a1, r),
                  __shfl_sync(~0u, own.b1, r)};
    };
    const Span sa = row_of(g), sb = row_of(g + 8), hl = hull_of(row_of(0), row_of(15));

    // pages of 8-key groups: lane 2 t + i holds group i of unit t of a batch of 16
    const int* table = a.table + seq * a.table_stride;
    auto entry = [&](int batch) -> int {  // -1 where none is needed or it is no page
      const int u = batch * 16 + (lane >> 1);
      if (u >= n) return -1;
      const int j = un.first_key(u0 + u) + warp * kSlice + (lane & 1) * 8;
      if (!span_hits(hl, j, j + 8)) return -1;
      const int p = __ldg(table + j / a.page_size);
      if (p < 0 || p >= a.n_pages) {
        paged_report(a.status, kStatusDeviceArg, 51);
        return -1;
      }
      return p;
    };
    // a lane copies 16 bytes of every fourth key of a group
    const uint8_t* const k_lane = static_cast<const uint8_t*>(a.kc) + head * a.head_stride + (lane >> 3) * a.token_stride + (lane & 7) * 16;
    const long long to_v = static_cast<const char*>(a.vc) - static_cast<const char*>(a.kc);
    const uint8_t* const s_lane = ((lane & 2) ? a.vs : a.ks) + head * a.scale_head_stride;
    uint32_t place[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = 4 * i + (lane >> 3);
      place[i] = key * 128 + (((lane & 7) ^ swizzle8(key)) << 4);
    }
    int page_now = -1, page_next = entry(0), in_page = 0;
    auto issue = [&](int u) {  // copies the warp's keys of unit u into stage u % kStages8
      if (u < n) {
        if ((u & 15) == 0) {
          page_now = page_next;
          const int v = u + (lane >> 1);
          in_page = v < n ? (un.first_key(u0 + v) + warp * kSlice + (lane & 1) * 8) % a.page_size : 0;
          page_next = entry((u >> 4) + 1);
        }
        const int j0 = un.first_key(u0 + u) + warp * kSlice;
        const bool all = span_covers(hl, j0, j0 + kSlice);
        if (all || span_hits(hl, j0, j0 + kSlice)) {
          const uint32_t dst = ring + (u % kStages8) * kStage8;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int page = __shfl_sync(~0u, page_now, 2 * (u & 15) + i), in = __shfl_sync(~0u, in_page, 2 * (u & 15) + i);
            const uint8_t* src = k_lane + max(page, 0) * a.page_stride + in * a.token_stride;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t bytes = page >= 0 && (all || in_span(hl, j0 + 8 * i + 4 * k + (lane >> 3))) ? 16u : 0u;
              cp_async_16(dst + i * 1024 + place[k], src, bytes);
              cp_async_16(dst + i * 1024 + place[k] + kSlice8, src + to_v, bytes);
              src += 4 * a.token_stride;
            }
            // lanes i (K) and i + 2 (V): the group's factors
            if (lane < 4 && (lane & 1) == i)
              cp_async_8(dst + 2 * kSlice8 + (lane >> 1) * kSlice + i * 8, s_lane + max(page, 0) * a.scale_page_stride + in, page >= 0 ? 8u : 0u);
          }
        }
      }
      cp_async_commit();
    };
    uint32_t qa[8][4];
    float fa, fb;  // scores of row ra are fa times the products with q's fp16 form
    {
      const T* q = static_cast<const T*>(a.q);
      uint32_t lo[8], hi[8];
      int e = load_q(q + (sg.q_off + ra / a.G) * a.q_stride + (head * a.G + ra % a.G) * kHeadDim, c, lo, hi);
      fa = ldexpf(a.scale_log2, e);
#pragma unroll
      for (int s = 0; s < 8; ++s) qa[s][0] = lo[s], qa[s][2] = hi[s];
      e = load_q(q + (sg.q_off + rb / a.G) * a.q_stride + (head * a.G + rb % a.G) * kHeadDim, c, lo, hi);
      fb = ldexpf(a.scale_log2, e);
#pragma unroll
      for (int s = 0; s < 8; ++s) qa[s][1] = lo[s], qa[s][3] = hi[s];
    }
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    const uint32_t k_at = g * 128 + ((c ^ swizzle8(g)) << 4);  // key g, piece c; piece c + 4 differs in one bit
    uint32_t v_at[2];                                          // keys 2 c and 2 c + 1, piece g
#pragma unroll
    for (int i = 0; i < 2; ++i) v_at[i] = (2 * c + i) * 128 + ((g ^ swizzle8(2 * c + i)) << 4);
#pragma unroll 1
    for (int u = -2; u < n; ++u) {
      issue(u + 2);
      if (u < 0) continue;
      cp_async_wait<2>();
      __syncwarp();
      const int j0 = un.first_key(u0 + u) + warp * kSlice;
      if (!span_hits(hl, j0, j0 + kSlice)) continue;
      const uint32_t sk = ring + (u % kStages8) * kStage8, sv = sk + kSlice8, sf = sv + kSlice8;
      float s[2][4] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = lds16(sk + t * 1024 + (k_at ^ (h << 6)));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            warp_mma(s[t], qa[4 * h + k], e4m3x2_to_f16x2(word(x, k)), e4m3x2_hi_to_f16x2(word(x, k)), __half());
        }
      // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the slice: exponents of their factors
      float ek[4], ev[4], vi[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t bk = lds_u16(sf + 8 * t + 2 * c), bv = lds_u16(sf + kSlice + 8 * t + 2 * c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ek[2 * t + i] = two_to(factor_of((bk >> (8 * i)) & 0xFFu));
          const int e = factor_of((bv >> (8 * i)) & 0xFFu);
          ev[2 * t + i] = static_cast<float>(e);
          vi[2 * t + i] = two_to(-e);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[t][e] = fmaf(s[t][e] * ek[2 * t + (e & 1)], e < 2 ? fa : fb, ev[2 * t + (e & 1)]);
      const bool part = !__all_sync(~0u, span_covers(sa, j0, j0 + kSlice) && span_covers(sb, j0, j0 + kSlice));
      if (part) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + 8 * t + 2 * c + (e & 1);
            if (!in_span(e < 2 ? sa : sb, j)) s[t][e] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
        mx[r] = fmaxf(__fadd_ru(mx[r], -12.f), m[r]);
      }
      if (__any_sync(~0u, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = mx[r] > m[r] ? ex2_approx(m[r] - mx[r]) : 1.f;
          m[r] = mx[r];
          l[r] *= f;
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            o[t][2 * r] *= f;
            o[t][2 * r + 1] *= f;
          }
        }
      }
      uint32_t p[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[r] == -INFINITY ? 0.f : m[r];
        float e[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w = ex2_approx(s[t][2 * r + i] - base);
            e[2 * t + i] = w;
            l[r] = fmaf(w, vi[2 * t + i], l[r]);
          }
        p[r] = Half2<__half>::pack(e[0], e[1]);
        p[2 + r] = Half2<__half>::pack(e[2], e[3]);
      }
      // rows of V: keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9, columns 16 g to 16 g + 15
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lds16(sv + (i >> 1) * 1024 + v_at[i & 1]);
      if (part) {
        // NaN in a key that some row does not attend must not meet a weight of
        // 0: it is taken out, and added where the key is attended
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) bad |= e4m3_nan(word(v[i], k));
        if (__any_sync(~0u, bad)) hide_nan(v, sv, j0, sa, sb, o);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a0 = __byte_perm(word(v[0], k), word(v[1], k), 0x5140), a1 = __byte_perm(word(v[0], k), word(v[1], k), 0x7362);
        const uint32_t b0 = __byte_perm(word(v[2], k), word(v[3], k), 0x5140), b1 = __byte_perm(word(v[2], k), word(v[3], k), 0x7362);
        warp_mma(o[4 * k], p, e4m3x2_to_f16x2(a0), e4m3x2_to_f16x2(b0), __half());
        warp_mma(o[4 * k + 1], p, e4m3x2_hi_to_f16x2(a0), e4m3x2_hi_to_f16x2(b0), __half());
        warp_mma(o[4 * k + 2], p, e4m3x2_to_f16x2(a1), e4m3x2_to_f16x2(b1), __half());
        warp_mma(o[4 * k + 3], p, e4m3x2_hi_to_f16x2(a1), e4m3x2_hi_to_f16x2(b1), __half());
      }
      __syncwarp();  // the stage is refilled by the next issue
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
    }
    cp_async_wait<0>();
    __syncwarp();
    float* po = reinterpret_cast<float*>(ring_);  // [16][132], now that the ring is empty
    // o[t][0], o[t][1]: row g, columns 32 c + t and 32 c + 16 + t
#pragma unroll
    for (int t = 0; t < 16; t += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(po + (g + 8 * (e >> 1)) * 132 + 32 * c + 16 * (e & 1) + t) =
            make_float4(o[t][e], o[t + 1][e], o[t + 2][e], o[t + 3][e]);
    if (c == 0) {
      m_out[g] = m[0];
      m_out[g + 8] = m[1];
      l_out[g] = l[0];
      l_out[g + 8] = l[1];
    }
  }

  // NaN of the slice's rows of V: zero in v, and added to the sums of the rows
  // that attend its key (a positive weight times NaN is NaN; so no weight is
  // needed).
  static __device__ __forceinline__ void hide_nan(uint4 (&v)[4], uint32_t sv, int j0, const Span& sa, const Span& sb, float (&o)[16][4]) {
    const int c = threadIdx.x & 3;
    auto clear = [](uint32_t& w) { w &= ~((e4m3_nan(w) >> 7) * 0xFFu); };
#pragma unroll
    for (int i = 0; i < 4; ++i) clear(v[i].x), clear(v[i].y), clear(v[i].z), clear(v[i].w);
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll 1
    for (int k = 0; k < kSlice; ++k) {
      const bool ta = in_span(sa, j0 + k), tb = in_span(sb, j0 + k);
      // this lane's columns of key k: pieces 2 c and 2 c + 1
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = lds16(sv + k * 128 + (((2 * c + i) ^ swizzle8(k & 7)) << 4));
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const bool is = ((word(x, t >> 2) >> (8 * (t & 3))) & 0x7Fu) == 0x7Fu;
          if (is && ta) o[t][i] = nan;
          if (is && tb) o[t][2 + i] = nan;
        }
      }
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kDecThreads, 2)
    paged_decode8_kernel(const __grid_constant__ PagedAttnArgs a, bool behind) {
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ DecodeShared sh;
  launch_dependents();
  decode_span<Worker8<T>>(a, sh, ring, behind);
  clear_unowned_rows(a);
  if (behind) grid_wait();
}

template <typename T>
cudaError_t launch_decode(const PagedAttnArgs& a, bool behind, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_decode8_kernel<T>, kFewSmem8, done);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_after(paged_decode8_kernel<T>, dim3(std::min(2 * num_sms, kPagedMaxCtas)), kDecThreads, kFewSmem8, st, a,
                      behind);
}

}  // namespace

void launch_paged_write8(const PagedWrite8Args& a, bool fp16, int num_sms, cudaStream_t st) {
  const long long n = (static_cast<long long>(a.n_rows) * a.Hkv * 16 + 255) / 256;
  if (n == 0) return;
  const int grid = static_cast<int>(std::min<long long>(n, num_sms * 8LL));
  note_launches(1);
  if (fp16)
    paged_write8_kernel<__half><<<grid, 256, 0, st>>>(a);
  else
    paged_write8_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
}

void launch_paged_read8(const PagedRead8Args& a, bool fp16, int num_sms, cudaStream_t st) {
  const long long n = (static_cast<long long>(a.n) * a.page_size * a.Hkv * 8 + 255) / 256;
  if (n == 0) return;
  const int grid = static_cast<int>(std::min<long long>(n, num_sms * 8LL));
  note_launches(1);
  if (fp16)
    paged_read8_kernel<__half><<<grid, 256, 0, st>>>(a);
  else
    paged_read8_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
}

cudaError_t launch_paged_decode8(const PagedAttnArgs& a, bool behind, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch_decode<__half>(a, behind, num_sms, st) : launch_decode<__nv_bfloat16>(a, behind, num_sms, st);
}

}  // namespace lca
