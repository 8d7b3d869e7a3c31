// lca_paged8.cu — kernels of the 8-bit paged cache: quantising new keys and
// values into their pages, reading pages back, and attention of few rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lca_paged.cuh"
#include "lca_paged8.cuh"
#include "lca_paged_few.cuh"
#include "sm103.cuh"

namespace lca {
namespace {

// ------------------------------------------------------------------ write
// 8 threads per (row, head), for K and V together: each reads 32 bytes of both,
// the quarter-warp finds the two rows' largest magnitudes (as integers: a positive
// float's bits are in its order), and each thread writes 16 bytes of both.  The factor is a power of two, so dividing by
// it is an exact product and the only rounding is e4m3's.  Reads 512 bytes a
// row and head and writes 258.
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

// 16 values; v8: by one load, the address being a multiple of 32.
__device__ __forceinline__ void load32(const uint16_t* p, bool v8, uint4 (&x)[2]) {
  if (v8) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x), "=r"(x[1].y), "=r"(x[1].z), "=r"(x[1].w)
        : "l"(p));
  } else {
    x[0] = __ldg(reinterpret_cast<const uint4*>(p));
    x[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
}

// Largest magnitude of 16 values, as the type's bits; with kFinite of those
// that are finite.
template <typename T, bool kFinite>
__device__ __forceinline__ uint32_t largest(const uint4& x, const uint4& y) {
  uint32_t m = 0;
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    m = __vmaxu2(m, kFinite ? a & __vcmpltu2(a, Magnitude<T>::kInf) : a);
  }
  return max(m & 0xFFFFu, m >> 16);
}

// The smallest e with 2^e 448 >= m, as far as factors go: 448 = 1.75 2^8.
__device__ __forceinline__ int row_factor(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleMin), kScaleMax);
}

// Eight values over 2^e.  An infinity would end at 448: with kAll (some value of
// the row is not finite) it becomes NaN, so that it is not lost.
template <typename T, bool kAll>
__device__ __forceinline__ uint2 quantise(const uint4& x, int e) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
  if (!kAll && std::is_same<T, __half>::value && e >= -15 && e <= 14) {
    // a product of pairs, exact but for results below 2^-14, which become 0 either way
    const uint32_t h = static_cast<uint32_t>(15 - e) << 10;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = f16x2_to_e4m3x2(hmul2(w[i], h | h << 16));
  } else {
    const float f = two_to(-e), nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = Half2<T>::unpack(w[i]);
      r[i] = kAll ? to_e4m3x2(fabsf(v.x) == INFINITY ? nan : v.x * f, fabsf(v.y) == INFINITY ? nan : v.y * f)
                  : to_e4m3x2(v.x * f, v.y * f);
    }
  }
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}

// A quarter-warp takes kHeads heads of a row, so that as many loads of K and of V are
// under way and the slot is looked up once: 16.5K fp16 rows of 8 heads 17.1 us with
// two each, 17.8 with four; bf16 rows, tokens outermost, 16.0 (6.4 TB/s, 0.94 of a
// copy's rate) and 16.9.  Few rows take one each: the latency of more would show (64
// rows 2.4 us).  Before, instructions were the bound: with half-warps, 16 bytes a
// thread and four heads 19.2 us, and 21.3 while every value was looked at for being
// finite (now only where the row's largest says that some is not) and fp16 was
// scaled value by value.
template <typename T, int kHeads>
__global__ void __launch_bounds__(256) paged_write8_kernel(const PagedWrite8Args a) {
  const int groups = (a.Hkv + kHeads - 1) / kHeads;
  const long long n = static_cast<long long>(a.n_rows) * groups * 8;  // a multiple of 8: quarter-warps stay together
  const int piece = threadIdx.x & 7;
  const uint32_t quarter = 0xFFu << (threadIdx.x & 24);
  for (long long t = blockIdx.x * 256LL + threadIdx.x; t < n; t += gridDim.x * 256LL) {
    const long long row = line_div(t >> 3, groups);
    const int head0 = static_cast<int>((t >> 3) - row * groups) * kHeads;
    const int slot = __ldg(a.slots + row);
    if (slot < 0 || slot >= a.n_slots) continue;
    const int page = slot / a.page_size, token = slot % a.page_size;
    const uint16_t* k = a.k + row * a.k_stride + head0 * kHeadDim + piece * 16;
    const uint16_t* v = a.v + row * a.v_stride + head0 * kHeadDim + piece * 16;
    uint4 x[kHeads][2], y[kHeads][2];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (head0 + h < a.Hkv) {
        load32(k + h * kHeadDim, a.in_v8, x[h]);
        load32(v + h * kHeadDim, a.in_v8, y[h]);
      }
    int factor = 0;  // lane 2 h keeps K's of head h, lane 2 h + 1 V's
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (head0 + h >= a.Hkv) break;
      auto of_row = [&](uint32_t m) {
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(quarter, m, d));
        return m;
      };
      uint32_t m = of_row(largest<T, false>(x[h][0], x[h][1]) | largest<T, false>(y[h][0], y[h][1]) << 16);
      const bool all = __vcmpgeu2(m, Magnitude<T>::kInf) != 0;  // some value is not finite
      if (all) m = of_row(largest<T, true>(x[h][0], x[h][1]) | largest<T, true>(y[h][0], y[h][1]) << 16);
      const int ek = row_factor(Magnitude<T>::value(m & 0xFFFFu)), ev = row_factor(Magnitude<T>::value(m >> 16));
      const long long at = page * a.page_stride + token * a.token_stride + (head0 + h) * a.head_stride + piece * 16;
      auto put = [&](uint8_t* to, const uint4(&z)[2], int e) {
        const uint2 lo = all ? quantise<T, true>(z[0], e) : quantise<T, false>(z[0], e);
        const uint2 hi = all ? quantise<T, true>(z[1], e) : quantise<T, false>(z[1], e);
        *reinterpret_cast<uint4*>(to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      };
      put(a.kc + at, x[h], ek);
      put(a.vc + at, y[h], ev);
      if (piece >> 1 == h) factor = (piece & 1) ? ev : ek;
    }
    const int head = head0 + (piece >> 1);
    if (piece < 2 * kHeads && head < a.Hkv)
      ((piece & 1) ? a.vs : a.ks)[page * a.scale_page_stride + head * a.scale_head_stride + token] =
          static_cast<uint8_t>(factor + kScaleBias);
  }
}

// ------------------------------------------------------------------ read back
// 8 threads per row of K and V, 16 bytes of each read and 32 written, rows in
// the order in which they lie in the cache.  A block takes 32 kRows rows of a page
// at a time, each thread kRows of them, so that their loads are under way at
// once: 131K tokens of 8 heads 160 us one by one, 134 in fours, 150 in eights; and
// stores of 32 bytes take it to 126 (6.4 TB/s, 0.94 of a copy's rate).
// page_of(i, first) is the page whose copy page i of the result is (first: one thread asks
// so for each i); one that is none leaves it as it was.
template <typename T, int kRows, typename Page>
__device__ __forceinline__ void read_pages(const PagedRead8Args& a, Page page_of) {
  const unsigned rows = static_cast<unsigned>(a.page_size) * a.Hkv;  // of a page, below 2^31
  const unsigned parts = (rows + 32 * kRows - 1) / (32 * kRows);
  const long long n = static_cast<long long>(a.n) * parts;
  const int piece = threadIdx.x & 7;
  const unsigned inner = a.token_first ? a.page_size : a.Hkv;
  for (long long b = blockIdx.x; b < n; b += gridDim.x) {
    const long long i = line_div(b, parts);
    const unsigned row0 = static_cast<unsigned>(b - i * parts) * (32 * kRows) + (threadIdx.x >> 3);
    const int page = page_of(i, b == i * parts && threadIdx.x == 0);
    if (page < 0 || page >= a.n_pages) continue;
    uint4 x[kRows], y[kRows];
    uint32_t bk[kRows], bv[kRows];
    long long to[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const unsigned row = row0 + 32 * u, out = row / inner, in = row - out * inner;
      if (row >= rows) break;
      const int token = a.token_first ? in : out, head = a.token_first ? out : in;
      const long long at = page * a.page_stride + token * a.token_stride + head * a.head_stride + piece * 16;
      const long long st = page * a.scale_page_stride + head * a.scale_head_stride + token;
      to[u] = i * a.out_page_stride + token * a.out_token_stride + head * a.out_head_stride + piece * 16;
      x[u] = __ldg(reinterpret_cast<const uint4*>(a.kc + at));
      y[u] = __ldg(reinterpret_cast<const uint4*>(a.vc + at));
      bk[u] = __ldg(a.ks + st);
      bv[u] = __ldg(a.vs + st);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (row0 + 32 * u >= rows) break;
      auto put = [&](uint16_t* dst, const uint4& w, float f) {
        const uint2 p = Dequant<T>::quad(w.x, f), q = Dequant<T>::quad(w.y, f), r = Dequant<T>::quad(w.z, f),
                    s = Dequant<T>::quad(w.w, f);
        if (a.out_v8) {
          const uint32_t z[8] = {p.x, p.y, q.x, q.y, r.x, r.y, s.x, s.y};
          st_global_v8(dst, z);
        } else {
          *reinterpret_cast<uint4*>(dst) = make_uint4(p.x, p.y, q.x, q.y);
          *reinterpret_cast<uint4*>(dst + 8) = make_uint4(r.x, r.y, s.x, s.y);
        }
      };
      put(a.k + to[u], x[u], two_to(factor_of(bk[u])));
      put(a.v + to[u], y[u], two_to(factor_of(bv[u])));
    }
  }
}

template <typename T, int kRows>
__global__ void __launch_bounds__(256) paged_read8_kernel(const PagedRead8Args a) {
  read_pages<T, kRows>(a, [&](long long i, bool) { return __ldg(a.pages + i); });
}

// The same for the block tables of a batch (their entries one after another are
// the result's pages): of each request that the kernel for many rows serves the pages
// with keys that some of its rows attends.  map gets the result's tables, -1 for
// the others.
template <typename T, int kRows>
__global__ void __launch_bounds__(256)
    paged_copy8_kernel(const __grid_constant__ PagedRead8Args a, const __grid_constant__ PagedAttnArgs m, int* map) {
  read_pages<T, kRows>(a, [&](long long i, bool first) {
    const long long seq = line_div(i, m.max_pages);
    const int entry = static_cast<int>(i - seq * m.max_pages);
    int page = -1;
    const SegInfo sg = paged_seg(m, static_cast<int>(seq));
    if (sg.q_len > 0 && !few_rows(m, sg.q_len) && span_hits(hull(m, sg.q_len, sg.k_len, 0, sg.q_len), entry * m.page_size, (entry + 1) * m.page_size))
      page = __ldg(m.table + seq * m.table_stride + entry);
    if (first) map[i] = page >= 0 && page < a.n_pages ? static_cast<int>(i) : -1;
    return page;
  });
}

// ------------------------------------------------------------------ attention, few rows
// A warp's share of the line in lca_paged_few.cuh: a key costs 258 bytes, which
// bounds the work once the instructions that a key costs are few enough.
// Measured, whole calls: 64 requests of 1K-32K keys, 64 heads on 8, 198 us (6.0 TB/s,
// 0.89 of a copy's rate; 215 on another GPU), 32 of 2K-16K with 16 heads of their
// own, fp16, 138 us (5.9 TB/s), 4 of 512K 649 us (6.7 TB/s), one of 4K 15 us.  What
// is left of the first is rows of 128 bytes, tokens apart: with the tokens of a
// head together, 32 of 16K take 175 us where they take 193.
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
// product.  w is rounded to fp16 times 2^12 to 2^15: keys down to 2^-36 of the
// largest count, below 2^-26 with fewer bits.  The sums go by m, which was max -
// 12 when it was last set: it moves up (and the sums are rescaled) only once
// 2^15 would be passed.  It is rounded up, so that w stays in range where 12 is
// less than the last place of a huge score.
//
// Layout.  The keys are the rows of the products and the rows of q their
// columns: S^T = K q^T and O^T = V^T w^T, m16n8k16.  So a tile of 8 rows wastes
// nothing where 8 query heads share a KV head, and more of them share what a
// key's conversion costs: 32 requests of 1K-16K keys take 99 us with 16 rows, 127
// with 24, 157 with 32; with 40 their sums spill and they take 300, the kernel for
// many rows 172.  The operands K and V^T come from shared memory by 16-byte loads and are converted in
// registers.  The order of the 128 products of a score, and of the rows of O^T,
// is free, so a lane takes the bytes that lie together: of keys lane / 4 and 8
// more the pieces lane % 4 and lane % 4 + 4 (four values are two registers of one
// k16 step, q permuted to fit), and of its four keys' values the piece
// lane / 4, whose 16 columns are its two rows of eight m16 tiles.  Pieces are
// swizzled so that neither pattern has bank conflicts.  The weights come as
// (key, rows) and are needed as (row, keys): movmatrix.
constexpr int kStages8 = 2;
constexpr int kUnit8 = 128;                           // keys per unit
constexpr int kKeys8 = kUnit8 / kDecWarps;            // per warp and unit, two k16 steps of the product with V
constexpr int kSlice8 = kKeys8 * 128;                 // bytes of K or V
constexpr int kStage8 = 2 * kSlice8 + 2 * kKeys8;     // with the factors'
constexpr int kWarp8 = kStages8 * kStage8 > 16 * 132 * 4 ? kStages8 * kStage8 : 16 * 132 * 4;
static_assert(kKeys8 == 32 && kStage8 % 16 == 0, "four groups of 8 keys, two steps of 16");

__device__ __forceinline__ uint32_t swizzle8(int key) { return (key & 6) ^ ((key & 1) << 2); }

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t word(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }
// An 8 x 8 matrix of 16-bit values, a pair per lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A row of q for the k16 steps, fp16 of q times 2^-e; returns e.
template <typename T>
__device__ __forceinline__ int load_q(const T* row, int c, uint32_t (&q)[8][2]) {
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
  // the largest lands in [2^14, 2^15), in two steps: 2^-e itself may be past
  // a float's range
  const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 1) - 127 - 14;
  const float f0 = two_to(-e / 2), f1 = two_to(-e - -e / 2);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = Half2<T>::unpack(word(x[i], k));
      q[2 * i + (k >> 1)][k & 1] = Half2<__half>::pack(v.x * f0 * f1, v.y * f0 * f1);  // four values a step
    }
  return e;
}

// kTiles: tiles of 8 rows in an item.
template <typename T, int kTiles>
struct Worker8 {
  using Out = T;
  static constexpr int kRows = 8 * kTiles, kUnit = kUnit8;
  // Units per CTA 64: 64 requests of 1K-32K keys (83 units) 209 -> 199 us, 32 of
  // 16K (74) 188 -> 179, 256 of 1K (54) 100 -> 104 were they claimed.  One request of
  // 512K (8 heads) 193 -> 226 were its, in twice as many pieces; four 662 -> 651.
  static __device__ constexpr Claims claims() { return {64, 8, 1, 16}; }
  static constexpr int kWarpBytes = kWarp8 > kRows * 132 * 4 ? kWarp8 : kRows * 132 * 4;
  // With many tiles q does not fit the registers: it lies in shared memory for all
  // warps, and a unit's two steps of 16 keys go one after the other.
  static constexpr bool kShareQ = kTiles > 2;
  static constexpr int kSteps = kShareQ ? 1 : 2;
  static constexpr int kQBytes = kShareQ ? kTiles * (8 * 32 * 8 + 8 * 4) : 0;  // and a factor per row
  static constexpr float kBias = 0.f;
  static __device__ __forceinline__ void run(const PagedAttnArgs& a, uint8_t* ring_, int seq, const Request& sg,
                                             const Units& un, int tile, int head, int u0, int n, float* m_out, float* l_out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(ring_);
    const int r_first = tile * kRows;
    const int r_last = r_first + static_cast<int>(min(static_cast<long long>(sg.q_len) * a.G - r_first, static_cast<long long>(kRows))) - 1;
    // lane r finds row r's keys (a row past the last one repeats it, unused); hl: what some row attends
    const Span own = paged_span(a, sg.q_len, sg.k_len, min(r_first + lane % kRows, r_last) / a.G);
    auto row_of = [&](int r) {
      return Span{__shfl_sync(~0u, own.a0, r), __shfl_sync(~0u, own.b0, r), __shfl_sync(~0u, own.a1, r),
                  __shfl_sync(~0u, own.b1, r)};
    };
    const Span hl = hull_of(row_of(0), row_of(kRows - 1));

    // where 8-key groups lie: lane 4 t + i has group i of unit t of a batch of 8 units
    const int* table = a.table + seq * a.table_stride;
    auto key_of = [&](int batch) { return un.at(u0 + batch * 8 + (lane >> 2)) * kUnit8 + warp * kKeys8 + (lane & 3) * 8; };
    auto entry = [&](int batch) -> int {  // page, -1 where none is needed or it is no page
      if (batch * 8 + (lane >> 2) >= n) return -1;
      const int j = key_of(batch);
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
    const long long to_v = static_cast<const char*>(a.vc) - static_cast<const char*>(a.kc), step = 4 * a.token_stride;
    uint32_t place[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = 4 * i + (lane >> 3);
      place[i] = key * 128 + (((lane & 7) ^ swizzle8(key)) << 4);
    }
    int page_next = entry(0);
    long long off = -1, off_f = 0;  // of this lane's group: its first key, its factors
    auto issue = [&](int u) {       // copies the warp's keys of unit u into stage u % kStages8
      if (u < n) {
        if ((u & 7) == 0) {
          off = -1;
          if (page_next >= 0) {
            const int in = key_of(u >> 3) % a.page_size;
            off = page_next * a.page_stride + in * a.token_stride;
            off_f = page_next * a.scale_page_stride + head * a.scale_head_stride + in;
          }
          page_next = entry((u >> 3) + 1);
        }
        const int j0 = un.at(u0 + u) * kUnit8 + warp * kKeys8;
        const bool all = span_covers(hl, j0, j0 + kKeys8);
        if (all || span_hits(hl, j0, j0 + kKeys8)) {
          const uint32_t dst = ring + (u % kStages8) * kStage8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long base = __shfl_sync(~0u, off, 4 * (u & 7) + i);
            const uint8_t* src = k_lane + max(base, 0LL);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t bytes = base >= 0 && (all || in_span(hl, j0 + 8 * i + 4 * k + (lane >> 3))) ? 16u : 0u;
              cp_async_16(dst + i * 1024 + place[k], src, bytes);
              cp_async_16(dst + i * 1024 + place[k] + kSlice8, src + to_v, bytes);
              src += step;
            }
          }
          if ((lane >> 2) == (u & 7)) {
            const uint32_t bytes = off >= 0 ? 8u : 0u;
            cp_async_8(dst + 2 * kSlice8 + c * 8, a.ks + off_f, bytes);
            cp_async_8(dst + 2 * kSlice8 + kKeys8 + c * 8, a.vs + off_f, bytes);
          }
        }
      }
      cp_async_commit();
    };
    // q as B operands, and by what the products with a row's fp16 form give its scores
    uint32_t q[kShareQ ? 1 : kTiles][8][2];
    float f[kShareQ ? 1 : kTiles][2];
    const uint32_t shared_q = ring + (kDecWarps - warp) * kWarpBytes;
    const uint32_t shared_f = shared_q + kTiles * 8 * 32 * 8;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (kShareQ && t % kDecWarps != warp) continue;
      const int r = min(r_first + 8 * t + g, r_last), at = kShareQ ? 0 : t;
      const int e = load_q(static_cast<const T*>(a.q) + (sg.q_off + r / a.G) * a.q_stride + (head * a.G + r % a.G) * kHeadDim, c, q[at]);
      const float x = ldexpf(a.scale_log2, e);
      if constexpr (kShareQ) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sts64(shared_q + ((t * 8 + i) * 32 + lane) * 8, q[0][i][0], q[0][i][1]);
        if (c == 0) sts32(shared_f + (8 * t + g) * 4, __float_as_uint(x));
      } else {
        f[at][0] = __shfl_sync(~0u, x, 8 * c);
        f[at][1] = __shfl_sync(~0u, x, 8 * c + 4);
      }
    }
    if constexpr (kShareQ) __syncthreads();  // all warps have the same item
    float o[kTiles][8][4], m[kTiles][2], l[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }
    const uint32_t k_at = g * 128 + ((c ^ swizzle8(g)) << 4);  // key g, piece c; piece c + 4 differs in one bit
    uint32_t v_at[2];                                          // keys 2 c and 2 c + 1, piece g
#pragma unroll
    for (int i = 0; i < 2; ++i) v_at[i] = (2 * c + i) * 128 + ((g ^ swizzle8(2 * c + i)) << 4);
#pragma unroll 1
    for (int u = 1 - kStages8; u < n; ++u) {
      issue(u + kStages8 - 1);
      if (u < 0) continue;
      cp_async_wait<kStages8 - 1>();
      __syncwarp();
      const int j0 = un.at(u0 + u) * kUnit8 + warp * kKeys8;
      if (!span_hits(hl, j0, j0 + kKeys8)) continue;
      const uint32_t sk = ring + (u % kStages8) * kStage8, sv = sk + kSlice8, sf = sv + kSlice8;
      const bool part = !__all_sync(~0u, span_covers(own, j0, j0 + kKeys8));
#pragma unroll 1
      for (int b0 = 0; b0 < 2; b0 += kSteps) {
        // scores of keys 16 b + g (s[..][0], s[..][1]: the lane's two rows of a tile) and 16 b + g + 8
        float s[kSteps][kTiles][4];
#pragma unroll
        for (int b = 0; b < kSteps; ++b)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) s[b][t][0] = s[b][t][1] = s[b][t][2] = s[b][t][3] = 0.f;
#pragma unroll
        for (int b = 0; b < kSteps; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = sk + (b0 + b) * 2048 + (k_at ^ (h << 6));
            const uint4 x = lds16(at), y = lds16(at + 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w[4] = {e4m3x2_to_f16x2(word(x, k)), e4m3x2_to_f16x2(word(y, k)), e4m3x2_hi_to_f16x2(word(x, k)),
                                     e4m3x2_hi_to_f16x2(word(y, k))};
#pragma unroll
              for (int t = 0; t < kTiles; ++t) {
                uint2 z;
                if constexpr (kShareQ) {
                  z = lds64(shared_q + ((t * 8 + 4 * h + k) * 32 + lane) * 8);
                } else {
                  z = make_uint2(q[t][4 * h + k][0], q[t][4 * h + k][1]);
                }
                warp_mma(s[b][t], w, z.x, z.y, __half());
              }
            }
          }
        float vi[kSteps][2];  // 2^-ev
#pragma unroll
        for (int b = 0; b < kSteps; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = 16 * (b0 + b) + 8 * i + g;
            const float fk = two_to(factor_of(lds_u8(sf + key)));
            const int e = factor_of(lds_u8(sf + kKeys8 + key));
            vi[b][i] = two_to(-e);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              float2 ft;
              if constexpr (kShareQ) {
                const uint2 z = lds64(shared_f + (8 * t + 2 * c) * 4);
                ft = make_float2(__uint_as_float(z.x), __uint_as_float(z.y));
              } else {
                ft = make_float2(f[t][0], f[t][1]);
              }
              s[b][t][2 * i] = fmaf(s[b][t][2 * i] * fk, ft.x, static_cast<float>(e));
              s[b][t][2 * i + 1] = fmaf(s[b][t][2 * i + 1] * fk, ft.y, static_cast<float>(e));
            }
          }
        if (part) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const Span sp = row_of(8 * t + 2 * c + r);
#pragma unroll
              for (int b = 0; b < kSteps; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!in_span(sp, j0 + 16 * (b0 + b) + 8 * i + g)) s[b][t][2 * i + r] = -INFINITY;
            }
        }
        auto most = [&](int t, int r) {  // of this lane's keys
          float x = fmaxf(s[0][t][r], s[0][t][2 + r]);
          if constexpr (kSteps == 2) x = fmaxf(x, fmaxf(s[1][t][r], s[1][t][2 + r]));
          return x;
        };
        bool up = false;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) up |= __fadd_ru(most(t, r), -15.f) > m[t][r];
        if (__any_sync(~0u, up)) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float to = most(t, r);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) to = fmaxf(to, __shfl_xor_sync(~0u, to, d));
              to = __fadd_ru(to, -12.f);
              if (to > m[t][r]) {
                const float x = ex2_approx(m[t][r] - to);
                m[t][r] = to;
                l[t][r] *= x;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[t][i][r] *= x, o[t][i][2 + r] *= x;
              }
            }
        }
        uint32_t p[kSteps][kTiles][2];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const float b0_ = m[t][0] == -INFINITY ? 0.f : m[t][0], b1_ = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
          for (int b = 0; b < kSteps; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float w0 = ex2_approx(s[b][t][2 * i] - b0_), w1 = ex2_approx(s[b][t][2 * i + 1] - b1_);
              l[t][0] = fmaf(w0, vi[b][i], l[t][0]);
              l[t][1] = fmaf(w1, vi[b][i], l[t][1]);
              p[b][t][i] = transposed(Half2<__half>::pack(w0, w1));
            }
        }
#pragma unroll
        for (int b = 0; b < kSteps; ++b) {
          // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the step, columns 16 g to 16 g + 15
          const uint32_t sv_b = sv + (b0 + b) * 2048;
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = lds16(sv_b + (i >> 1) * 1024 + v_at[i & 1]);
          if (part) {
            // NaN in a key that some row does not attend must not meet a weight of
            // 0: it is taken out, and added where the key is attended
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) bad |= e4m3_nan(word(v[i], k));
            if (__any_sync(~0u, bad)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) finite(v[i].x), finite(v[i].y), finite(v[i].z), finite(v[i].w);
              // a positive weight times NaN is NaN, so no weight is needed
#pragma unroll 1
              for (int k = 0; k < 16; ++k) {
                const uint4 x = lds16(sv_b + k * 128 + ((g ^ swizzle8(k & 7)) << 4));
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    const Span sp = row_of(8 * t + 2 * c + r);
                    if (!in_span(sp, j0 + 16 * (b0 + b) + k)) continue;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      if ((e4m3_nan(word(x, i >> 2)) >> (8 * (i & 3) + 7)) & 1u) o[t][i >> 1][2 * (i & 1) + r] = __uint_as_float(0x7FC00000u);
                  }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // (column 4 k, 4 k + 1) of two keys each, then (4 k + 2, 4 k + 3)
            const uint32_t x0 = __byte_perm(word(v[0], k), word(v[1], k), 0x5140), x1 = __byte_perm(word(v[0], k), word(v[1], k), 0x7362);
            const uint32_t y0 = __byte_perm(word(v[2], k), word(v[3], k), 0x5140), y1 = __byte_perm(word(v[2], k), word(v[3], k), 0x7362);
            const uint32_t w0[4] = {e4m3x2_to_f16x2(x0), e4m3x2_hi_to_f16x2(x0), e4m3x2_to_f16x2(y0), e4m3x2_hi_to_f16x2(y0)};
            const uint32_t w1[4] = {e4m3x2_to_f16x2(x1), e4m3x2_hi_to_f16x2(x1), e4m3x2_to_f16x2(y1), e4m3x2_hi_to_f16x2(y1)};
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              warp_mma(o[t][2 * k], w0, p[b][t][0], p[b][t][1], __half());
              warp_mma(o[t][2 * k + 1], w1, p[b][t][0], p[b][t][1], __half());
            }
          }
        }
      }
      __syncwarp();  // the stage is refilled by the next issue
    }
    cp_async_wait<0>();
    __syncwarp();
    float* po = reinterpret_cast<float*>(ring_);  // [kRows][132], now that the ring is empty
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * t + 2 * c + r;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          *reinterpret_cast<float4*>(po + row * 132 + 16 * g + 2 * i) =
              make_float4(o[t][i][r], o[t][i][2 + r], o[t][i + 1][r], o[t][i + 1][2 + r]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][r] += __shfl_xor_sync(~0u, l[t][r], d);
        if (g == 0) {
          m_out[row] = m[t][r];
          l_out[row] = l[t][r];
        }
      }
  }

  static __device__ __forceinline__ void finite(uint32_t& w) { w &= ~((e4m3_nan(w) >> 7) * 0xFFu); }
};

// CTAs per SM: what registers and shared memory allow.
template <int kTiles>
constexpr int kPerSm = kTiles == 1 ? 3 : 2;

template <typename T, int kTiles>
__global__ void __launch_bounds__(kDecThreads, kPerSm<kTiles>)
    paged_decode8_kernel(const __grid_constant__ PagedAttnArgs a, bool behind) {
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ DecodeShared<8 * kTiles> sh;
  launch_dependents();
  decode_span<Worker8<T, kTiles>>(a, sh, ring, behind);
  clear_unowned_rows(a);
  if (behind) grid_wait();
}

template <typename T, int kTiles>
cudaError_t launch_decode(const PagedAttnArgs& a, bool behind, int num_sms, cudaStream_t st) {
  constexpr int kBytes = kDecWarps * Worker8<T, kTiles>::kWarpBytes + Worker8<T, kTiles>::kQBytes;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_decode8_kernel<T, kTiles>, kBytes, done);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_after(paged_decode8_kernel<T, kTiles>, dim3(std::min(kPerSm<kTiles> * num_sms, kPagedMaxCtas)), kDecThreads, kBytes,
                      st, a, behind);
}

template <typename T>
cudaError_t launch_decode_of(const PagedAttnArgs& a, int rows, bool behind, int num_sms, cudaStream_t st) {
  if (rows == 8) return launch_decode<T, 1>(a, behind, num_sms, st);
  if (rows == 16) return launch_decode<T, 2>(a, behind, num_sms, st);
  if (rows == 24) return launch_decode<T, 3>(a, behind, num_sms, st);
  return launch_decode<T, 4>(a, behind, num_sms, st);
}

}  // namespace

template <typename T>
void write8(const PagedWrite8Args& a, int num_sms, cudaStream_t st) {
  // two heads a quarter-warp where that still fills the GPU
  const long long one = static_cast<long long>(a.n_rows) * a.Hkv * 8;
  const bool many = a.Hkv >= 2 && one >= 2LL * 2048 * num_sms;
  const long long blocks = ((many ? static_cast<long long>(a.n_rows) * ((a.Hkv + 1) / 2) * 8 : one) + 255) / 256;
  const int grid = static_cast<int>(std::min<long long>(blocks, num_sms * 8LL));
  if (many)
    paged_write8_kernel<T, 2><<<grid, 256, 0, st>>>(a);
  else
    paged_write8_kernel<T, 1><<<grid, 256, 0, st>>>(a);
}

void launch_paged_write8(const PagedWrite8Args& a, bool fp16, int num_sms, cudaStream_t st) {
  note_launches(1);
  if (fp16)
    write8<__half>(a, num_sms, st);
  else
    write8<__nv_bfloat16>(a, num_sms, st);
}

void launch_paged_copy8(const PagedRead8Args& a, const PagedAttnArgs& m, int* map, bool fp16, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.page_size) * a.Hkv;
  const int grid = static_cast<int>(std::min<long long>(a.n * ((rows + 127) / 128), num_sms * 8LL));
  note_launches(1);
  if (fp16)
    paged_copy8_kernel<__half, 4><<<grid, 256, 0, st>>>(a, m, map);
  else
    paged_copy8_kernel<__nv_bfloat16, 4><<<grid, 256, 0, st>>>(a, m, map);
}

template <typename T>
void read8(const PagedRead8Args& a, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.page_size) * a.Hkv;
  // four rows a thread where that still fills the GPU
  if (a.n * rows * 8 >= 4LL * 2048 * num_sms)
    paged_read8_kernel<T, 4><<<static_cast<int>(std::min<long long>(a.n * ((rows + 127) / 128), num_sms * 8LL)), 256, 0, st>>>(a);
  else
    paged_read8_kernel<T, 1><<<static_cast<int>(std::min<long long>(a.n * ((rows + 31) / 32), num_sms * 8LL)), 256, 0, st>>>(a);
}

void launch_paged_read8(const PagedRead8Args& a, bool fp16, int num_sms, cudaStream_t st) {
  note_launches(1);
  if (fp16)
    read8<__half>(a, num_sms, st);
  else
    read8<__nv_bfloat16>(a, num_sms, st);
}

cudaError_t launch_paged_decode8(const PagedAttnArgs& a, int rows, bool behind, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch_decode_of<__half>(a, rows, behind, num_sms, st)
              : launch_decode_of<__nv_bfloat16>(a, rows, behind, num_sms, st);
}

}  // namespace lca
