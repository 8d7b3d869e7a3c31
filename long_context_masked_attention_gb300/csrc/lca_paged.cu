// lca_paged.cu — kernels of the paged cache: the batch plan, the writing of
// new keys and values into their pages, and attention over the pages.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lca_paged.cuh"
#include "lca_paged.h"
#include "sm103.cuh"

namespace lca {
namespace {

// ------------------------------------------------------------------ batch plan
// Two exclusive sums over the requests (new tokens; pages they need) place
// every row and every fresh page.  What bounds the call is latency, not its
// few bytes, so it is one launch without a second pass: each block runs the
// sums over all requests itself, 1024 at a time, and from each such tile
// writes only its own share of the rows and of the fresh pages (256 at a
// time, round robin), finding a row's request by bisection in shared memory.
// 6.2 us for 8 requests of a token each, 8.3 for 1024 requests with 61K rows
// (a replayed graph): latency in both.
constexpr int kPlanThreads = 1024;
constexpr int kPlanShare = 256;

// Inclusive sum over the block of a pair of 64-bit values.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, a, d), y = __shfl_up_sync(~0u, b, d);
    if (lane >= d) a += x, b += y;
  }
  if (lane == 31) part[warp][0] = a, part[warp][1] = b;
  __syncthreads();
  if (warp == 0) {
    long long x = part[lane][0], y = part[lane][1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(~0u, x, d), w = __shfl_up_sync(~0u, y, d);
      if (lane >= d) x += u, y += w;
    }
    part[lane][0] = x, part[lane][1] = y;
  }
  __syncthreads();
  if (warp > 0) a += part[warp - 1][0], b += part[warp - 1][1];
}

// Largest s in [0, n) with start[s] <= x.
__device__ __forceinline__ int bisect(const long long* start, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// tokens and page_size below 2^31
__device__ __forceinline__ int pages_of(unsigned tokens, unsigned page_size) {
  return static_cast<int>((tokens + page_size - 1) / page_size);
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedPlanArgs a) {
  __shared__ long long part[32][2];
  __shared__ long long row0[kPlanThreads + 1], page0[kPlanThreads + 1];  // exclusive sums of the tile
  __shared__ int ctx_s[kPlanThreads];
  const int tid = threadIdx.x;
  const long long room = static_cast<long long>(a.max_pages) * a.page_size;
  const unsigned page_size = a.page_size;
  const int taken = min(max(a.taken[0], 0), a.n_free);
  long long rows = 0, pages = 0;  // sums before the tile
  int bad = 0;
  for (int base = 0; base < a.n_seq; base += kPlanThreads) {
    const int n = min(kPlanThreads, a.n_seq - base);
    long long nw = 0, fresh = 0, ctx = 0, want_len = 0;
    int wrong = 0;
    if (tid < n) {
      const int c = a.ctx_len[base + tid], w = a.new_len[base + tid];
      nw = max(w, 0);
      ctx = min(static_cast<long long>(max(c, 0)), room);
      want_len = min(ctx + nw, room);
      wrong = c < 0 || w < 0 || c > room || ctx + nw > room;
      fresh = max(pages_of(static_cast<unsigned>(want_len), page_size) - pages_of(static_cast<unsigned>(ctx), page_size), 0);
    }
    long long ir = nw, ip = fresh;
    block_scan2(ir, ip, part);
    if (tid < n) {
      row0[tid] = rows + ir - nw;
      page0[tid] = pages + ip - fresh;
      ctx_s[tid] = static_cast<int>(ctx);
      if (rows + ir > a.n_rows) wrong = 1;
      if (blockIdx.x == 0) {
        if (base == 0 && tid == 0) a.q_start[0] = 0;
        a.q_start[base + tid + 1] = static_cast<int>(min(rows + ir, static_cast<long long>(a.n_rows)));
        a.k_len[base + tid] = static_cast<int>(want_len);
      }
    }
    if (tid == n - 1) row0[n] = rows + ir, page0[n] = pages + ip;
    bad += __syncthreads_count(wrong);

    // this block's share of the tile's rows
    const long long r_end = min(row0[n], static_cast<long long>(a.n_rows));
    const int sub = tid / kPlanShare, in = tid % kPlanShare;
    constexpr int kSubs = kPlanThreads / kPlanShare;
    const long long step = static_cast<long long>(gridDim.x) * kSubs, me = blockIdx.x * kSubs + sub;
    for (long long s = rows / kPlanShare + (me - rows / kPlanShare % step + step) % step; s * kPlanShare < r_end;
         s += step) {
      const long long r = s * kPlanShare + in;
      if (r < rows || r >= r_end) continue;
      const int i = bisect(row0, n, r);
      const long long at = ctx_s[i] + (r - row0[i]);
      const unsigned pos = static_cast<unsigned>(min(at, 0x7FFFFFFFLL));
      int slot = -1;
      if (at < room) {  // room < 2^31
        const unsigned c = pos / page_size;
        const int have = pages_of(ctx_s[i], page_size);
        int page;
        if (static_cast<int>(c) < have) {
          page = a.block_table[(base + i) * a.table_stride + c];
        } else {
          const long long f = taken + page0[i] + (static_cast<int>(c) - have);
          page = f < a.n_free ? a.free_pages[f] : -1;
        }
        if (page >= 0 && page < a.n_pages) slot = page * a.page_size + static_cast<int>(pos - c * page_size);
      }
      a.slots[r] = slot;
      a.positions[r] = static_cast<int>(pos);
    }
    // and of its fresh pages
    for (long long s = pages / kPlanShare + (me - pages / kPlanShare % step + step) % step; s * kPlanShare < page0[n];
         s += step) {
      const long long f = s * kPlanShare + in;
      if (f < pages || f >= page0[n]) continue;
      const int i = bisect(page0, n, f);
      const int have = pages_of(ctx_s[i], page_size);
      int page = taken + f < a.n_free ? a.free_pages[taken + f] : -1;
      if (page < 0 || page >= a.n_pages) page = -1;
      a.block_table[(base + i) * a.table_stride + have + (f - page0[i])] = page;
    }
    rows = row0[n];
    pages = page0[n];
    __syncthreads();  // the tile's arrays are reused
  }
  // rows behind the last request
  const long long first = min(rows, static_cast<long long>(a.n_rows));
  for (long long r = first + blockIdx.x * static_cast<long long>(kPlanThreads) + tid; r < a.n_rows;
       r += static_cast<long long>(gridDim.x) * kPlanThreads) {
    a.slots[r] = -1;
    a.positions[r] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (a.n_seq == 0) a.q_start[0] = 0;
    const long long left = a.n_free - taken;
    a.state[0] = static_cast<int>(taken + min(pages, left));
    a.state[1] = static_cast<int>(min(max(pages - left, 0LL), 0x7FFFFFFFLL));
    a.state[2] = bad;
    a.state[3] = static_cast<int>(first);
  }
}

// ------------------------------------------------------------------ write
// Copies 16-byte pieces: 16 threads per (row, head) for K and V together, so
// that a half-warp's loads and stores are the 256 contiguous bytes of a row
// whatever the strides between rows, heads and pages.  Bound by HBM: 16.5K rows
// of 8 heads take 22.6 us (6.0 TB/s, 0.88 of a copy's rate); 64 rows take 4.1.
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedWriteArgs a) {
  const long long n = static_cast<long long>(a.n_rows) * a.Hkv * 16;
  for (long long t = blockIdx.x * 256LL + threadIdx.x; t < n; t += gridDim.x * 256LL) {
    const int piece = static_cast<int>(t & 15);
    const long long rh = t >> 4;
    const int head = static_cast<int>(rh % a.Hkv);
    const long long row = rh / a.Hkv;
    const int slot = __ldg(a.slots + row);
    if (slot < 0 || slot >= a.n_slots) continue;
    const uint4 x = a.k[row * a.k_stride + head * 16 + piece], y = a.v[row * a.v_stride + head * 16 + piece];
    const long long at = slot / a.page_size * a.page_stride + slot % a.page_size * a.token_stride +
                         head * a.head_stride + piece;
    a.kc[at] = x;
    a.vc[at] = y;
  }
}

// ------------------------------------------------------------------ attention, few rows
// Attention is bound here by reading K and V once: with G query heads per KV
// head and t new tokens a request has G t rows per KV head, and 16 of them
// take part in every product, so a key costs 512 bytes from HBM and little
// arithmetic.  The work is a line of units of 64 keys (request, KV head, row
// tile, unit) cut into equal spans, one per CTA, two CTAs per SM, whatever
// the lengths; of a long line the last part is cut finer and claimed by the
// CTAs that are done first, since SMs differ in what they get of HBM.  A
// piece of an item that goes on in another span leaves unnormalised sums (O,
// running maximum, sum of exponentials) in the workspace, and the CTA that
// finishes an item's last piece joins them in the order of the keys.  Each CTA
// finds its span itself from the lengths, so there is no planning launch.
// Within a CTA each of 4 warps owns 16 of a unit's 64 keys,
// copies them asynchronously into its own ring of shared memory (keys that no
// row attends are filled with zeros, not read) and keeps its own running
// maximum and sums; the warps meet once per piece.  16 rows cannot fill a
// tcgen05 tile of 128, so the products are warp-wide m16n8k16 ones, whose
// score accumulators are already the A operand of the product with V.
// Measured (replayed graphs): 64 requests of 1K-32K keys, 64 query heads on 8,
// 364 us (6.5 TB/s, 0.96 of a copy's rate); 4 of 512K 1246 us (6.9 TB/s); 32 of
// 2K-16K with 16 heads of their own 249 us (6.5 TB/s); one of 4K 18.5 us, which
// is latency: start-up, keys and the join of the pieces.
constexpr int kUnit = 64;                     // keys per unit
constexpr int kRows = 16;                     // rows per item
constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kSlice = kUnit / kDecWarps;     // keys per warp and unit
constexpr int kDecStages = 3;
constexpr int kSliceBytes = kSlice * 256;     // of K or V
constexpr int kWarpBytes = kDecStages * 2 * kSliceBytes;
constexpr int kDecSmem = kDecWarps * kWarpBytes;
// Units per CTA from which on the line's last eighth is claimed.  Above it: 64
// requests of 1K-32K (1.1M keys) 698 -> 668 us, 4 of 512K 1293 -> 1248.  Below
// it the finer spans cost more than they even out: 256 requests of 1K, 134
// units per CTA, 185 us unclaimed and 196 claimed.
constexpr int kLongShare = 160;
// What an item costs beside its units, in units; 0 against 4: 128 requests of
// 100-8K keys 317.5 and 315.5 us, 64 of 500 43.4 and 43.1, 8 of 4K 43.2 and 39.7.
constexpr int kItemUnits = 4;
// A CTA's share, where there is that much; 2, 4 and 8: one request of 1K 14.5,
// 16.5 and 19.5 us, one of 4K 19.1, 18.5 and 20.5.
constexpr int kMinUnits = 4;
constexpr int kSeqTile = 2 * kDecThreads;     // requests whose places on the line are in shared memory at once
constexpr int kPartFloats = kRows * (kHeadDim + 2);
static_assert(kSlice == 16, "a slice is one k16 step of the product with V");
static_assert(kPartFloats == kPagedPartFloats, "workspace layout");

// The products take 16-bit operands, so p is rounded to the type (by 2^-8 of it
// at most in bf16, 2^-11 in fp16); l sums it unrounded.  Against 64 bits the
// largest error of O is 0.0023 (bf16) and 0.00027 (fp16) on normal values, where
// a p of 32 bits leaves 0.0017 and 0.00021, O's own rounding; products of 32-bit
// values would run at a fraction of the rate.
// bf16 has the exponents of fp32.  fp16 holds nothing below 2^-24: p, at most
// 1, is kept times 2^12, so that keys down to 2^-36 of the largest still
// count (below 2^-26 as subnormal numbers, with fewer bits); O, l and their
// partial sums carry the factor, the quotient and the LSE do not.
template <typename T>
constexpr float kBias = 0.f;
template <>
constexpr float kBias<__half> = 12.f;

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

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes, of which those past `bytes` (0 or 16) are zero
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The units of a hull: n0 from t0 on, then n1 from t1 on.
struct Units {
  int t0, n0, t1, n1;
  __device__ __forceinline__ int first_key(int u) const { return (u < n0 ? t0 + u : t1 + u - n0) * kUnit; }
};
__device__ __forceinline__ Units units_of(const Span& h) {
  Units u;
  u.t0 = h.a0 / kUnit;
  u.n0 = h.b0 > h.a0 ? (h.b0 + kUnit - 1) / kUnit - u.t0 : 0;
  u.t1 = max(h.a1 / kUnit, u.n0 > 0 ? u.t0 + u.n0 : 0);
  u.n1 = h.b1 > h.a1 ? max((h.b1 + kUnit - 1) / kUnit - u.t1, 0) : 0;
  return u;
}

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

struct DecodeShared {
  long long start[kSeqTile + 1];  // first unit of each request of the tile, relative to the tile's
  Request req[kSeqTile];
  long long sums[kDecWarps];
  float m[kDecWarps][kRows], l[kDecWarps][kRows];
  int last, next;
};

// Places of the requests [base, base + kSeqTile) on the line; returns their units.
__device__ __forceinline__ long long place_requests(const PagedAttnArgs& a, DecodeShared& sh, int base) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();  // earlier readers
  long long n0 = 0, mine = 0;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int i = base + 2 * tid + k;
    if (i >= a.n_seq) break;
    const SegInfo sg = paged_seg(a, i);
    if (sg.q_len > 0 && few_rows(a, sg.q_len)) {
      const Units u = units_of(hull(a, sg.q_len, sg.k_len, 0, sg.q_len));
      mine += static_cast<long long>(row_tiles(a, sg.q_len)) * a.Hkv * (max(u.n0 + u.n1, 1) + kItemUnits);
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
// share is long, two more per CTA over the rest.
struct Spans {
  long long total, big;
  int first, rest;
  __device__ __forceinline__ Spans(long long t, int grid) : total(t) {
    first = static_cast<int>(min(static_cast<long long>(grid), max(total / kMinUnits, 1LL)));
    rest = total / first >= kLongShare ? 2 * first : 0;
    big = rest > 0 ? total - total / 8 : total;
  }
  __device__ __forceinline__ long long start(int c) const {
    return c <= first ? line_div(c * big, first) : big + line_div((c - first) * (total - big), rest);
  }
  __device__ __forceinline__ int of(long long p) const {
    return static_cast<int>(p < big ? line_div((p + 1) * first - 1, big)
                                    : first + line_div((p - big + 1) * rest - 1, total - big));
  }
};

// One warp's share of a piece: units [u0, u0 + n) of an item, keys
// [16 warp, 16 warp + 16) of each.
template <typename T>
struct WarpState {
  float o[16][4];  // rows lane / 4 and lane / 4 + 8, columns 8 t + 2 (lane % 4), + 1
  float m[2], l[2];
};

template <typename T>
__device__ __forceinline__ void decode_warp(const PagedAttnArgs& a, uint32_t ring, int seq, const Request& sg,
                                            const Units& un, int tile, int head, int u0, int n, WarpState<T>& st) {
  using H = Half2<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(static_cast<int>(min(static_cast<long long>(sg.q_len) * a.G - tile * kRows, 16LL)), kRows);
  const int r_first = tile * kRows, r_last = r_first + rows - 1;
  // the two rows of this lane (a row past the last one repeats it, unused)
  const int ra = min(r_first + (lane >> 2), r_last), rb = min(r_first + (lane >> 2) + 8, r_last);
  // lane r finds row r's keys; hl: what some row attends
  const Span own = paged_span(a, sg.q_len, sg.k_len, min(r_first + (lane & 15), r_last) / a.G);
  auto row_of = [&](int r) {
    return Span{__shfl_sync(~0u, own.a0, r), __shfl_sync(~0u, own.b0, r), __shfl_sync(~0u, own.a1, r),
                __shfl_sync(~0u, own.b1, r)};
  };
  const Span sa = row_of(lane >> 2), sb = row_of((lane >> 2) + 8), hl = hull_of(row_of(0), row_of(15));

  // offsets of 8-key groups: lane 2 t + g holds group g of unit t of a batch of 16
  const int* table = a.table + seq * a.table_stride;
  auto entry = [&](int batch) -> int {  // page of this lane's group, -1 where none is needed or it is no page
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
  auto offset = [&](int batch, int page) -> long long {
    if (page < 0) return -1;
    const int j = un.first_key(u0 + batch * 16 + (lane >> 1)) + warp * kSlice + (lane & 1) * 8;
    return page * a.page_stride + j % a.page_size * a.token_stride;
  };
  // a lane copies 16 bytes of every second key of a group: its first key's
  // address, the step to the next, the places in the stage
  const T* const k_lane =
      static_cast<const T*>(a.kc) + head * a.head_stride + (lane >> 4) * a.token_stride + (lane & 15) * 8;
  const long long to_v = static_cast<const char*>(a.vc) - static_cast<const char*>(a.kc), step = 2 * a.token_stride;
  uint32_t place[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    place[i] = (2 * i + (lane >> 4)) * 256 + (((lane & 15) ^ (2 * i + (lane >> 4))) << 4);
  int page_next = entry(0);
  long long off = 0;
  // copies the warp's keys of unit u into stage u % 3
  auto issue = [&](int u) {
    if (u < n) {
      if ((u & 15) == 0) {
        off = offset(u >> 4, page_next);
        page_next = entry((u >> 4) + 1);
      }
      const int j0 = un.first_key(u0 + u) + warp * kSlice;
      const bool all = span_covers(hl, j0, j0 + kSlice);  // no key to leave out
      if (all || span_hits(hl, j0, j0 + kSlice)) {
        const uint32_t dst = ring + (u % kDecStages) * 2 * kSliceBytes;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const long long base = __shfl_sync(~0u, off, 2 * (u & 15) + g);
          const T* src = k_lane + max(base, 0LL);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t bytes = base >= 0 && (all || in_span(hl, j0 + 8 * g + 2 * i + (lane >> 4))) ? 16u : 0u;
            cp_async_16(dst + g * 2048 + place[i], src, bytes);
            cp_async_16(dst + g * 2048 + place[i] + kSliceBytes, reinterpret_cast<const char*>(src) + to_v, bytes);
            src += step;
          }
        }
      }
    }
    cp_async_commit();
  };
  // Q as A operands, straight from global memory
  uint32_t q[8][4];
  {
    const T* q0 = static_cast<const T*>(a.q);
    const T* pa = q0 + (sg.q_off + ra / a.G) * a.q_stride + (head * a.G + ra % a.G) * kHeadDim + 2 * (lane & 3);
    const T* pb = q0 + (sg.q_off + rb / a.G) * a.q_stride + (head * a.G + rb % a.G) * kHeadDim + 2 * (lane & 3);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      q[c][0] = __ldg(reinterpret_cast<const uint32_t*>(pa + 16 * c));
      q[c][1] = __ldg(reinterpret_cast<const uint32_t*>(pb + 16 * c));
      q[c][2] = __ldg(reinterpret_cast<const uint32_t*>(pa + 16 * c + 8));
      q[c][3] = __ldg(reinterpret_cast<const uint32_t*>(pb + 16 * c + 8));
    }
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) st.o[t][0] = st.o[t][1] = st.o[t][2] = st.o[t][3] = 0.f;
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;

  // this lane's row and 16-byte column of the four 8x8 matrices of ldmatrix
  const int kkey = (lane & 7) + ((lane >> 4) << 3), kcol = (lane >> 3) & 1;   // K: (keys 0-7, 8-15) x (d 0-7, 8-15)
  const int vkey = (lane & 7) + (((lane >> 3) & 1) << 3), vcol = lane >> 4;   // V, transposed
#pragma unroll 1
  for (int u = -2; u < n; ++u) {
    issue(u + 2);  // two units ahead
    if (u < 0) continue;
    cp_async_wait<2>();
    __syncwarp();
    const int j0 = un.first_key(u0 + u) + warp * kSlice;
    if (!span_hits(hl, j0, j0 + kSlice)) continue;
    const uint32_t sk = ring + (u % kDecStages) * 2 * kSliceBytes, sv = sk + kSliceBytes;
    float s[2][4] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t b[4];
      ldsm4(b, sk + kkey * 256 + (((2 * c + kcol) ^ (kkey & 7)) << 4));
      warp_mma(s[0], q[c], b[0], b[1], T());
      warp_mma(s[1], q[c], b[2], b[3], T());
    }
    const bool part = !__all_sync(~0u, span_covers(sa, j0, j0 + kSlice) && span_covers(sb, j0, j0 + kSlice));
    if (part) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 8 * t + 2 * (lane & 3) + (e & 1);
          if (!in_span(e < 2 ? sa : sb, j)) s[t][e] = -INFINITY;
        }
    }
    float mx[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])) * a.scale_log2;
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
      mx[r] = fmaxf(mx[r], st.m[r]);
    }
    if (__any_sync(~0u, mx[0] > st.m[0] || mx[1] > st.m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = mx[r] > st.m[r] ? ex2_approx(st.m[r] - mx[r]) : 1.f;
        st.m[r] = mx[r];
        st.l[r] *= f;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          st.o[t][2 * r] *= f;
          st.o[t][2 * r + 1] *= f;
        }
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float base = (st.m[r] == -INFINITY ? 0.f : st.m[r]) - kBias<T>;
      float e[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        e[2 * t] = ex2_approx(fmaf(s[t][2 * r], a.scale_log2, -base));
        e[2 * t + 1] = ex2_approx(fmaf(s[t][2 * r + 1], a.scale_log2, -base));
      }
      st.l[r] += (e[0] + e[1]) + (e[2] + e[3]);
      p[r] = H::pack(e[0], e[1]);
      p[2 + r] = H::pack(e[2], e[3]);
    }
    bool alone = false;
    if (part) {
      // a value that is not finite, in keys that some row does not attend?
      uint32_t bad = 0;
#pragma unroll 1
      for (int t = 0; t < 8; ++t) {
        uint32_t b[4];
        ldsm4t(b, sv + vkey * 256 + (((2 * t + vcol) ^ (vkey & 7)) << 4));
        bad |= H::not_finite(b[0]) | H::not_finite(b[1]) | H::not_finite(b[2]) | H::not_finite(b[3]);
      }
      alone = __any_sync(~0u, bad & 0x80008000u);
    }
    if (!alone) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        uint32_t b[4];
        ldsm4t(b, sv + vkey * 256 + (((2 * t + vcol) ^ (vkey & 7)) << 4));
        warp_mma(st.o[2 * t], p, b[0], b[1], T());
        warp_mma(st.o[2 * t + 1], p, b[2], b[3], T());
      }
    } else {
      // 0 times such a value would be NaN: each row adds its own keys only
#pragma unroll 1
      for (int k = 0; k < kSlice; ++k) {
        const int from = (lane & ~3) | ((k & 7) >> 1);
        const float2 x0 = H::unpack(__shfl_sync(~0u, k < 8 ? p[0] : p[2], from));
        const float2 x1 = H::unpack(__shfl_sync(~0u, k < 8 ? p[1] : p[3], from));
        const float pa = (k & 1) ? x0.y : x0.x, pb = (k & 1) ? x1.y : x1.x;
        const bool ta = in_span(sa, j0 + k), tb = in_span(sb, j0 + k);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          uint32_t w;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(sv + k * 256 + ((t ^ (k & 7)) << 4) + 4 * (lane & 3)));
          const float2 vv = H::unpack(w);
          if (ta) {
            st.o[t][0] = fmaf(pa, vv.x, st.o[t][0]);
            st.o[t][1] = fmaf(pa, vv.y, st.o[t][1]);
          }
          if (tb) {
            st.o[t][2] = fmaf(pb, vv.x, st.o[t][2]);
            st.o[t][3] = fmaf(pb, vv.y, st.o[t][3]);
          }
        }
      }
    }
    __syncwarp();  // the stage is refilled by the next issue
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    st.l[r] += __shfl_xor_sync(~0u, st.l[r], 1);
    st.l[r] += __shfl_xor_sync(~0u, st.l[r], 2);
  }
}

template <typename T>
__device__ __forceinline__ void st_row16(T* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = Half2<T>::pack(x[2 * k], x[2 * k + 1]);
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
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

template <typename T>
__device__ __forceinline__ void decode_span(const PagedAttnArgs& a, DecodeShared& sh, uint8_t* ring, bool behind) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // requests whose rows do not overlap make fewer than 2^52 units; a q_start
  // that lets them overlap may make more, and is reported and not served then
  constexpr long long kMost = 1LL << 52;
  long long total = 0;
  for (int base = 0; base < a.n_seq; base += kSeqTile)
    total = min(total + place_requests(a, sh, base), kMost);
  if (!behind) grid_wait();  // counts and status are cleared
  if (total == 0 || total == kMost) return;
  const Spans sp(total, gridDim.x);
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
      tile1 += place_requests(a, sh, base);
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
    const int tiles = row_tiles(a, sg.q_len);
    const int head = static_cast<int>(line_div(item, tiles));
    const int tile = static_cast<int>(item - static_cast<long long>(head) * tiles);

    const int rows = static_cast<int>(min(static_cast<long long>(sg.q_len) * a.G - static_cast<long long>(tile) * kRows,
                                          static_cast<long long>(kRows)));
    float* po = reinterpret_cast<float*>(ring + warp * kWarpBytes);  // [16][132], once the ring is empty
    {
      WarpState<T> st;
      // an item without keys has one unit that holds none
      decode_warp<T>(a, smem_u32(po), seq, sg, un, tile, head, u0, un.n0 + un.n1 > 0 ? n : 0, st);
      cp_async_wait<0>();
      __syncwarp();
      const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        *reinterpret_cast<float2*>(po + r * 132 + 8 * t + c) = make_float2(st.o[t][0], st.o[t][1]);
        *reinterpret_cast<float2*>(po + (r + 8) * 132 + 8 * t + c) = make_float2(st.o[t][2], st.o[t][3]);
      }
      if ((lane & 3) == 0) {
        sh.m[warp][r] = st.m[0];
        sh.m[warp][r + 8] = st.m[1];
        sh.l[warp][r] = st.l[0];
        sh.l[warp][r + 8] = st.l[1];
      }
    }
    __syncthreads();
    const int row = tid >> 3, col = (tid & 7) * 16;
    // the four warps' sums of row `row`, columns col .. col + 15
    float m = -INFINITY, l = 0.f, x[16] = {};
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, sh.m[w][row]);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float f = sh.l[w][row] != 0.f ? ex2_approx(sh.m[w][row] - m) : 0.f;
      l = fmaf(f, sh.l[w][row], l);
      const float* pw = reinterpret_cast<const float*>(ring + w * kWarpBytes) + row * 132 + col;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(pw + 4 * k);
        x[4 * k] = fmaf(f, y.x, x[4 * k]);
        x[4 * k + 1] = fmaf(f, y.y, x[4 * k + 1]);
        x[4 * k + 2] = fmaf(f, y.z, x[4 * k + 2]);
        x[4 * k + 3] = fmaf(f, y.w, x[4 * k + 3]);
      }
    }
    if (n < nu) {
      // first and last span of the item; span c's first piece is in slot 2 c
      // and a later, unfinished one in slot 2 c + 1
      const int c0 = sp.of(i0), c1 = sp.of(i0 + nu - 1);
      const int late = sp.start(c0) < i0 - kItemUnits ? 1 : 0;
      auto slot = [&](int c) { return a.parts + (2 * c + (c == c0 ? late : 0)) * static_cast<long long>(kPartFloats); };
      float* part = slot(span);
      if (row < rows) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          __stcg(reinterpret_cast<float4*>(part + row * kHeadDim + col) + k,
                 make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]));
        if ((tid & 7) == 0) {
          __stcg(part + kRows * kHeadDim + row, m);
          __stcg(part + kRows * kHeadDim + kRows + row, l);
        }
      }
      __syncthreads();
      if (tid == 0) {  // its fences cover what the barrier has ordered before and after them
        __threadfence();
        sh.last = atomicAdd(a.arrived + c0, 1) == c1 - c0;
        __threadfence();
      }
      __syncthreads();
      if (sh.last) {
        auto piece = [&](int k) {
          return a.parts + (2 * (c0 + k) + (k == 0 ? late : 0)) * static_cast<long long>(kPartFloats);
        };
#pragma unroll 1
        for (int i = 2 * warp; i < rows; i += 2 * kDecWarps) {
          float mr, lr, y[2][4];
          join_rows<kRows, 2, 8>(c1 - c0 + 1, piece, i, mr, lr, y);
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
                    lk == 0.f ? -INFINITY : (mk + log2f(lk) - kBias<T>) * 0.6931471805599453f;
            }
          }
        }
      }
    } else if (row < rows) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] *= inv;
      const long long r = static_cast<long long>(tile) * kRows + row;
      const long long token = sg.q_off + r / a.G;
      const int h = head * a.G + static_cast<int>(r % a.G);
      st_row16(static_cast<T*>(a.o) + (token * a.Hq + h) * kHeadDim + col, x);
      if ((tid & 7) == 0)
        a.lse[static_cast<long long>(h) * a.Tq + token] =
            l == 0.f ? -INFINITY : (m + log2f(l) - kBias<T>) * 0.6931471805599453f;
    }
    __syncthreads();  // the ring is refilled
  }
}

// behind: launched under the kernel for many rows, which lets this one start
// once the call's first kernel has ended; this one's CTAs then take the SMs
// that the other leaves, and end only after it, so that what follows them in
// the stream waits for both.
template <typename T>
__global__ void __launch_bounds__(kDecThreads, 2)
    paged_decode_kernel(const __grid_constant__ PagedAttnArgs a, bool behind) {
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ DecodeShared sh;
  launch_dependents();
  decode_span<T>(a, sh, ring, behind);
  clear_unowned_rows(a);
  if (behind) grid_wait();
}

}  // namespace

void launch_paged_plan(const PagedPlanArgs& a, int num_sms, cudaStream_t st) {
  // a block per 1024 rows, one each for its threads: the sums are the same
  // work for one block or for all of them at once.  61K rows with a block per
  // 512, 1024, 2048 and 4096 of them: 8.35, 8.4, 10.3 and 12.4 us
  const int grid = std::max(1, std::min(num_sms, static_cast<int>((static_cast<long long>(a.n_rows) + 1023) / 1024)));
  note_launches(1);
  paged_plan_kernel<<<grid, kPlanThreads, 0, st>>>(a);
}

void launch_paged_write(const PagedWriteArgs& a, int num_sms, cudaStream_t st) {
  const long long n = (static_cast<long long>(a.n_rows) * a.Hkv * 16 + 255) / 256;
  if (n == 0) return;
  note_launches(1);
  paged_write_kernel<<<static_cast<int>(std::min<long long>(n, num_sms * 8LL)), 256, 0, st>>>(a);
}

template <typename T>
cudaError_t launch_decode(const PagedAttnArgs& a, bool behind, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_decode_kernel<T>, kDecSmem, done);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_after(paged_decode_kernel<T>, dim3(std::min(2 * num_sms, kPagedMaxCtas)), kDecThreads, kDecSmem, st, a,
                      behind);
}

cudaError_t launch_paged_decode(const PagedAttnArgs& a, bool behind, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch_decode<__half>(a, behind, num_sms, st) : launch_decode<__nv_bfloat16>(a, behind, num_sms, st);
}

}  // namespace lca
