// lca_paged_few.cuh — attention of few rows over a paged cache: the line of
// work that the kernels for 16-bit and for 8-bit caches share, how CTAs share it
// and how its pieces are joined.  The kernels bring what a warp does with its keys.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lca_paged.cuh"
#include "lca_paged.h"
#include "sm103.cuh"

namespace lca {
namespace {

// Attention is bound here by reading K and V once: with G query heads per KV
// head and t new tokens a request has G t rows per KV head, and a tile of them
// takes part in every product, so a key costs its bytes from HBM and little
// arithmetic.  The work is a line of units of keys (request, KV head, row
// tile, unit) cut into equal spans, one per CTA, a few CTAs per SM, whatever
// the lengths; of a long line the last part is cut finer and claimed by the
// CTAs that are done first, since SMs differ in what they get of HBM.  A
// piece of an item that goes on in another span leaves unnormalised sums (O,
// running maximum, sum of exponentials) in the workspace, and the CTA that
// finishes an item's last piece joins them in the order of the keys.  Each CTA
// finds its span itself from the lengths, so there is no planning launch.
// Within a CTA each of 4 warps owns a quarter of a unit's keys and keeps its own
// running maximum and sums; the warps meet once per piece.
//
// A worker W says what a warp does with its share of a piece, and how many rows
// an item and keys a unit have (W::kRows, W::kUnit).  The constants'
// measurements are of 16-bit caches, whose units of 64 keys are 32 KB; those of an
// 8-bit cache have 128 keys and as many bytes.
constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
// How the last part of a long line is claimed: from `share` units per CTA on,
// one in `part` of it, in `spans` spans per CTA.  For a 16-bit cache, above it:
// 64 requests of 1K-32K (1.1M keys) 698 -> 668 us, 4 of 512K 1293 -> 1248.  Below
// it the finer spans cost more than they even out: 256 requests of 1K, 134
// units per CTA, 185 us unclaimed and 196 claimed.  Not where an item would have
// more than `pieces` pieces, which one CTA joins.
struct Claims {
  int share, part, spans, pieces;
};
// What an item costs beside its units, in units; 0 against 4: 128 requests of
// 100-8K keys 317.5 and 315.5 us, 64 of 500 43.4 and 43.1, 8 of 4K 43.2 and 39.7.
constexpr int kItemUnits = 4;
// A CTA's share, where there is that much; 2, 4 and 8: one request of 1K 14.5,
// 16.5 and 19.5 us, one of 4K 19.1, 18.5 and 20.5.
constexpr int kMinUnits = 4;
constexpr int kSeqTile = 2 * kDecThreads;     // requests whose places on the line are in shared memory at once

__device__ __forceinline__ void warp_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         __nv_bfloat16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void warp_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes, of which those past `bytes` (0 or 16) are zero
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The units of a hull: n0 from t0 on, then n1 from t1 on.
struct Units {
  int t0, n0, t1, n1;
  __device__ __forceinline__ int at(int u) const { return u < n0 ? t0 + u : t1 + u - n0; }
};
template <int kUnit>
__device__ __forceinline__ Units units_of(const Span& h) {
  Units u;
  u.t0 = h.a0 / kUnit;
  u.n0 = h.b0 > h.a0 ? (h.b0 + kUnit - 1) / kUnit - u.t0 : 0;
  u.t1 = max(h.a1 / kUnit, u.n0 > 0 ? u.t0 + u.n0 : 0);
  u.n1 = h.b1 > h.a1 ? max((h.b1 + kUnit - 1) / kUnit - u.t1, 0) : 0;
  return u;
}

template <int kRows>
__device__ __forceinline__ int row_tiles(const PagedAttnArgs& a, int q_len) {
  return static_cast<int>((static_cast<long long>(q_len) * a.G + kRows - 1) / kRows);
}

// A request as the line has it: every (row tile, KV head) has kItemUnits and
// then the units of the whole request's hull, at least one, so that rows
// without keys are written.
struct Request {
  int q_off, q_len, k_len;
  Units un;
};

template <int kRows>
struct DecodeShared {
  long long start[kSeqTile + 1];  // first unit of each request of the tile, relative to the tile's
  Request req[kSeqTile];
  long long sums[kDecWarps];
  float m[kDecWarps][kRows], l[kDecWarps][kRows];
  int last, next;
};

// Places of the requests [base, base + kSeqTile) on the line; returns their units.
template <typename W>
__device__ __forceinline__ long long place_requests(const PagedAttnArgs& a, DecodeShared<W::kRows>& sh, int base) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();  // earlier readers
  long long n0 = 0, mine = 0;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int i = base + 2 * tid + k;
    if (i >= a.n_seq) break;
    const SegInfo sg = paged_seg(a, i);
    if (sg.q_len > 0 && few_rows(a, sg.q_len)) {
      const Units u = units_of<W::kUnit>(hull(a, sg.q_len, sg.k_len, 0, sg.q_len));
      mine += static_cast<long long>(row_tiles<W::kRows>(a, sg.q_len)) * a.Hkv * (max(u.n0 + u.n1, 1) + kItemUnits);
      sh.req[2 * tid + k] = Request{sg.q_off, sg.q_len, sg.k_len, u};
    }
    if (k == 0) n0 = mine;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) sh.sums[warp] = inc;
  __syncthreads();
  long long at = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) at += sh.sums[w];
    total += sh.sums[w];
  }
  sh.start[2 * tid] = at;
  sh.start[2 * tid + 1] = at + n0;
  if (tid == kDecThreads - 1) sh.start[kSeqTile] = total;
  __syncthreads();
  return total;
}

// The line's spans: one per CTA over its first `big` units and, where a CTA's
// share is long, some more per CTA over the rest.
struct Spans {
  long long total, big;
  int first, rest;
  __device__ __forceinline__ Spans(long long t, int grid, long long heads, Claims c) : total(t) {
    first = static_cast<int>(min(static_cast<long long>(grid), max(total / kMinUnits, 1LL)));
    rest = total / first >= c.share && first / c.pieces <= heads ? c.spans * first : 0;
    big = rest > 0 ? total - total / c.part : total;
  }
  __device__ __forceinline__ long long start(int c) const {
    return c <= first ? line_div(c * big, first) : big + line_div((c - first) * (total - big), rest);
  }
  __device__ __forceinline__ int of(long long p) const {
    return static_cast<int>(p < big ? line_div((p + 1) * first - 1, big)
                                    : first + line_div((p - big + 1) * rest - 1, total - big));
  }
};

template <typename T, int N>
__device__ __forceinline__ void st_row(T* dst, const float (&x)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 8)
    *reinterpret_cast<uint4*>(dst + k) =
        make_uint4(Half2<T>::pack(x[k], x[k + 1]), Half2<T>::pack(x[k + 2], x[k + 3]), Half2<T>::pack(x[k + 4], x[k + 5]),
                   Half2<T>::pack(x[k + 6], x[k + 7]));
}

// o = 0, lse = -inf in the rows [r0, r1), by all CTAs.
__device__ __noinline__ void clear_rows(const PagedAttnArgs& a, int r0, int r1) {
  const long long n = static_cast<long long>(r1 - r0) * a.Hq * 16;
  for (long long t = blockIdx.x * static_cast<long long>(kDecThreads) + threadIdx.x; t < n;
       t += gridDim.x * static_cast<long long>(kDecThreads)) {
    const unsigned rh = static_cast<unsigned>(t >> 4);  // Tq Hq < 2^31
    const unsigned h = rh % a.Hq;
    const long long row = r0 + static_cast<long long>(rh / a.Hq);
    reinterpret_cast<uint4*>(a.o)[(row * a.Hq + h) * 16 + (t & 15)] = make_uint4(0, 0, 0, 0);
    if ((t & 15) == 0) a.lse[static_cast<long long>(h) * a.Tq + row] = -INFINITY;
  }
}

// Rows outside every request, and rows of a request behind its last key.
__device__ __forceinline__ void clear_unowned_rows(const PagedAttnArgs& a) {
  const SegInfo s0 = a.n_seq > 0 ? paged_rows(a, 0) : SegInfo{};
  const SegInfo s1 = a.n_seq > 0 ? paged_rows(a, a.n_seq - 1) : SegInfo{};
  clear_rows(a, 0, s0.q_off);
  clear_rows(a, s1.q_off + s1.q_len, a.Tq);
  if (!a.ctx_len) return;
  for (int base = 0; base < a.n_seq; base += kDecThreads) {
    const int i = base + threadIdx.x;
    if (!__syncthreads_or(i < a.n_seq && paged_seg(a, i).q_len < paged_rows(a, i).q_len)) continue;
    for (int k = base; k < min(base + kDecThreads, a.n_seq); ++k) {
      const SegInfo s = paged_seg(a, k);
      clear_rows(a, s.q_off + s.q_len, s.q_off + paged_rows(a, k).q_len);
    }
  }
}

// The line's work of this CTA.  W::run takes units [u0, u0 + n) of an item, this
// warp's keys of each, through its W::kWarpBytes of shared memory, and leaves
// there the sums of the rows as [W::kRows][132] floats, and in m and l their maxima
// and sums of exponentials.  W::Out is o's type; the sums carry a factor of 2^W::kBias.
template <typename W>
__device__ __forceinline__ void decode_span(const PagedAttnArgs& a, DecodeShared<W::kRows>& sh, uint8_t* ring, bool behind) {
  using T = typename W::Out;
  constexpr int kRows = W::kRows, kPartFloats = kRows * (kHeadDim + 2);
  constexpr int kAtOnce = kRows < 16 ? kRows : 16;  // rows that the CTA's threads take at a time,
  constexpr int kCols = kAtOnce;                    // so many columns each
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // requests whose rows do not overlap make fewer than 2^52 units; a q_start
  // that lets them overlap may make more, and is reported and not served then
  constexpr long long kMost = 1LL << 52;
  long long total = 0;
  for (int base = 0; base < a.n_seq; base += kSeqTile)
    total = min(total + place_requests<W>(a, sh, base), kMost);
  if (!behind) grid_wait();  // counts and status are cleared
  if (total == 0 || total == kMost) return;
  const Spans sp(total, gridDim.x, static_cast<long long>(a.n_seq) * a.Hkv, W::claims());
  if (blockIdx.x >= sp.first) return;
  int base = a.n_seq > kSeqTile ? -kSeqTile : 0;      // requests in sh.start begin at base
  long long tile0 = 0, tile1 = a.n_seq > kSeqTile ? 0 : total;  // their units
  int span = blockIdx.x;
  long long pos = sp.start(span), end = sp.start(span + 1);
  for (;;) {
    if (pos == end) {  // the next span that nobody has; spans are claimed in order, so it lies further on
      if (sp.rest == 0) return;
      if (tid == 0) sh.next = sp.first + atomicAdd(a.claims, 1);
      __syncthreads();
      span = sh.next;
      if (span >= sp.first + sp.rest) return;
      pos = sp.start(span);
      end = sp.start(span + 1);
      __syncthreads();  // next is written again only after all have read it
      if (pos == end) continue;
    }
    while (pos >= tile1) {
      base += kSeqTile;
      if (base >= a.n_seq) return;  // only if the lengths changed meanwhile
      tile0 = tile1;
      tile1 += place_requests<W>(a, sh, base);
    }
    int lo = 0, hi = min(kSeqTile, a.n_seq - base);  // the last request that starts at or before pos
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.start[mid] <= pos - tile0) lo = mid; else hi = mid;
    }
    const int seq = base + lo;
    const Request sg = sh.req[lo];
    const Units un = sg.un;
    const int nu = max(un.n0 + un.n1, 1);
    const long long local = pos - tile0 - sh.start[lo];
    const long long item = line_div(local, nu + kItemUnits);
    // the span has the item's places [from, to), of which the first kItemUnits hold no keys
    const int from = static_cast<int>(local - item * (nu + kItemUnits));
    const int to = from + static_cast<int>(min(static_cast<long long>(nu + kItemUnits - from), end - pos));
    const long long i0 = pos - from + kItemUnits;  // the item's first unit
    pos += to - from;
    const int u0 = max(from - kItemUnits, 0), n = to - kItemUnits - u0;
    if (n <= 0) continue;
    const int tiles = row_tiles<kRows>(a, sg.q_len);
    const int head = static_cast<int>(line_div(item, tiles));
    const int tile = static_cast<int>(item - static_cast<long long>(head) * tiles);

    const int rows = static_cast<int>(min(static_cast<long long>(sg.q_len) * a.G - static_cast<long long>(tile) * kRows,
                                          static_cast<long long>(kRows)));
    // an item without keys has one unit that holds none
    W::run(a, ring + warp * W::kWarpBytes, seq, sg, un, tile, head, u0, un.n0 + un.n1 > 0 ? n : 0, sh.m[warp],
           sh.l[warp]);
    __syncthreads();
    const bool cut = n < nu;
    int c0 = 0, c1 = 0, late = 0;
    if (cut) {
      // first and last span of the item; span c's first piece is in slot 2 c
      // and a later, unfinished one in slot 2 c + 1
      c0 = sp.of(i0), c1 = sp.of(i0 + nu - 1);
      late = sp.start(c0) < i0 - kItemUnits ? 1 : 0;
    }
    auto slot = [&](int c) { return a.parts + (2 * c + (c == c0 ? late : 0)) * static_cast<long long>(kPartFloats); };
    constexpr int kPer = kDecThreads / kAtOnce;  // threads per row
    const int col = tid % kPer * kCols;
#pragma unroll 1
    for (int row = tid / kPer; row < rows; row += kAtOnce) {
      // the four warps' sums of row `row`, columns col .. col + kCols - 1
      float m = -INFINITY, l = 0.f, x[kCols] = {};
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, sh.m[w][row]);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = sh.l[w][row] != 0.f ? ex2_approx(sh.m[w][row] - m) : 0.f;
        l = fmaf(f, sh.l[w][row], l);
        const float* pw = reinterpret_cast<const float*>(ring + w * W::kWarpBytes) + row * 132 + col;
#pragma unroll
        for (int k = 0; k < kCols / 4; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(pw + 4 * k);
          x[4 * k] = fmaf(f, y.x, x[4 * k]);
          x[4 * k + 1] = fmaf(f, y.y, x[4 * k + 1]);
          x[4 * k + 2] = fmaf(f, y.z, x[4 * k + 2]);
          x[4 * k + 3] = fmaf(f, y.w, x[4 * k + 3]);
        }
      }
      if (cut) {
        float* part = slot(span);
#pragma unroll
        for (int k = 0; k < kCols / 4; ++k)
          __stcg(reinterpret_cast<float4*>(part + row * kHeadDim + col) + k,
                 make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]));
        if (tid % kPer == 0) {
          __stcg(part + kRows * kHeadDim + row, m);
          __stcg(part + kRows * kHeadDim + kRows + row, l);
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
#pragma unroll
        for (int k = 0; k < kCols; ++k) x[k] *= inv;
        const long long r = static_cast<long long>(tile) * kRows + row;
        const long long token = sg.q_off + r / a.G;
        const int h = head * a.G + static_cast<int>(r % a.G);
        st_row(static_cast<T*>(a.o) + (token * a.Hq + h) * kHeadDim + col, x);
        if (tid % kPer == 0)
          a.lse[static_cast<long long>(h) * a.Tq + token] =
              l == 0.f ? -INFINITY : (m + log2f(l) - W::kBias) * 0.6931471805599453f;
      }
    }
    if (cut) {
      __syncthreads();
      if (tid == 0) {  // its fences cover what the barrier has ordered before and after them
        __threadfence();
        sh.last = atomicAdd(a.arrived + c0, 1) == c1 - c0;
        __threadfence();
      }
      __syncthreads();
      if (sh.last) {
#pragma unroll 1
        for (int i = 2 * warp; i < rows; i += 2 * kDecWarps) {
          float mr, lr, y[2][4];
          join_rows<kRows, 2, 8>(c1 - c0 + 1, [&](int k) { return slot(c0 + k); }, i, mr, lr, y);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mk = __shfl_sync(~0u, mr, 16 * k), lk = __shfl_sync(~0u, lr, 16 * k);
            if (i + k < rows) {
              const long long r = static_cast<long long>(tile) * kRows + i + k;
              const long long token = sg.q_off + r / a.G;
              const int h = head * a.G + static_cast<int>(r % a.G);
              const float inv = lk == 0.f ? 0.f : 1.f / lk;
              *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + (token * a.Hq + h) * kHeadDim + 4 * lane) =
                  make_uint2(Half2<T>::pack(y[k][0] * inv, y[k][1] * inv), Half2<T>::pack(y[k][2] * inv, y[k][3] * inv));
              if (lane == 0)
                a.lse[static_cast<long long>(h) * a.Tq + token] =
                    lk == 0.f ? -INFINITY : (mk + log2f(lk) - W::kBias) * 0.6931471805599453f;
            }
          }
        }
      }
    }
    __syncthreads();  // the ring is refilled
  }
}

}  // namespace
}  // namespace lca
