// lca_paged_chunk.cu — attention of many rows over a paged cache for sm_103a
// (tcgen05 + TMEM + TMA): prompts, chunks of prompts, drafts to verify.
//
// The rows of a request that share a KV head are packed: row t G + g of a
// head's block is new token t, query head g of the group, so the G query
// heads read every key once and a block of few tokens still fills a tile.  A
// sub-tile of 128 rows holds tpt = floor(128 / G) tokens; an item is two
// sub-tiles of one (request, KV head).  Queries come by TMA as boxes of
// [token][head of the group][64], keys and values as boxes of the rows of one
// page: gcd(page_size, 128) rows, so that no box leaves its page and a
// 128-key tile is a whole number of them whatever the page size.  Table
// entries are read by the producer's lanes one tile ahead; keys that no row
// attends are not read (a box outside the array is filled with zeros).
//
// The products bound the work (4 d operations per attended pair); per key
// tile and item 1024 keys' rows pass the tensor core against 64 KB of K and V
// from L2.  Roles as in the packed forward: warp 9 loads, warp 8 issues
// S = Q K^T and O += P V, warps 0-7 are two softmax warpgroups, each thread
// one row; warp 10 finds the next items and their key ranges ahead of them.
// The tiles of all items form one line that is cut into equal spans, one per
// CTA (paged_begin_kernel places the items on it), so that batches of any
// mixture of lengths end together; the items that a cut divides leave
// their sums in the workspace and paged_join_kernel joins them in the order
// of the keys.  An item of one sub-tile (a narrow one: at most 128 rows)
// gives both score buffers to that sub-tile, so that the product with the
// next keys runs while the first warpgroup works on the present ones.
//
// Measured (whole calls, replayed graphs, 64 query heads on 8): 2048 tokens at
// the end of 32K keys 1503-1641 us (1.38-1.51 PFLOP/s; the tensor pipe is active
// 64 % of the time, and power decides the rest); 8 prompts of 101-2047 tokens 284-295
// us, where an item of 9 tiles takes 18 us of which 14-15 are tiles; 5 tokens of
// each of 32 requests at 1K-16K keys 163 us (0.78 of a copy's rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lca_paged.cuh"
#include "lca_paged.h"
#include "sm103.cuh"

namespace lca {
namespace {

constexpr int kThreads = 352;
constexpr int kStages = 5;
constexpr uint32_t kTileBytes = 32768;   // 128 rows x 128 values
constexpr uint32_t kChunkBytes = 16384;  // 128 rows x 64 values, 128-byte swizzled
constexpr int kOffQ = 0;
constexpr int kOffKV = 2 * kTileBytes;
constexpr int kOffCtl = kOffKV + kStages * kTileBytes;
constexpr int kSmemBytes = kOffCtl + 1024 + 1024;
constexpr int kItemSlots = 3;
// A CTA's share, where there is that much; 2, 4 and 8: a chunk of 509 tokens
// with a window of 1024 beside 15 single tokens 62.2, 62.3 and 64.1 us.
constexpr int kMinTiles = 4;
// What an item costs beside its tiles, in tiles; 3, 4, 5 and 6: 32 requests of
// 5 tokens at 1K-16K keys 173, 173.3, 175.6 and 176.4 us, 8 prompts of 101-2047
// 209, 206, 209 and 216.
constexpr int kItemCost = 3;

// Scores and probabilities have three barriers each: those of sub-tiles 0 and
// 1, and one for the odd tiles of a narrow item, which go through sub-tile
// 1's columns to the first warpgroup.  So each barrier has one waiting
// warpgroup, which sees all of its phases: a wait by parity must not be two
// phases behind.
enum : int {
  B_QFULL = 0,
  B_QEMPTY = 1,
  B_KVFULL = 2,
  B_KVEMPTY = B_KVFULL + kStages,
  B_SFULL = B_KVEMPTY + kStages,
  B_PFULL = B_SFULL + 3,
  B_OFULL = B_PFULL + 3,
  B_ITFULL = B_OFULL + 2,
  B_ITEMPTY = B_ITFULL + kItemSlots,
  B_DRAIN = B_ITEMPTY + kItemSlots,
  B_COUNT = B_DRAIN + 1
};

// What the scheduler tells the other roles about a piece of an item.
struct Item {
  int valid, narrow;
  int n, u0;              // its tiles: u0 .. u0 + n - 1 of the item's
  int head, tok0;         // KV head; first token, inside the request
  int part;               // workspace slot of its sums, -1 when it is the whole item
  int seq;
  int q_off, q_len, k_len;
  int t0, n0, t1;         // the item's tiles: n0 from t0 on, then from t1 on
  int pad[2];
  Span hull[2], full[2];  // per sub-tile: keys that some, and that all, of its rows attend
  Span all, every;        // keys that some, and that all, of the item's rows attend
  __device__ __forceinline__ int tile(int t) const { return u0 + t < n0 ? t0 + u0 + t : t1 + u0 + t - n0; }
  __device__ __forceinline__ uint32_t cls(int x, int kt) const {
    const int j0 = kt * kTile;
    if (!span_hits(hull[x], j0, j0 + kTile)) return kTileEmpty;
    return span_covers(full[x], j0, j0 + kTile) ? kTileFull : kTilePartial;
  }
};
static_assert(sizeof(Item) == 160 && 8 * B_COUNT <= 256 && kItemSlots * sizeof(Item) <= 640,
              "the items lie between the barriers and the TMEM slot");

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// p is rounded to the type, as the products' operand (see lca_paged.cu).
// fp16 holds nothing below 2^-24 and p reaches 2^8 between rescalings, so p
// is kept times 2^7: at most 2^15, and keys down to 2^-31 of the largest count
// (below 2^-21 as subnormal numbers, with fewer bits).
template <typename T>
constexpr float kBias = 0.f;
template <>
constexpr float kBias<__half> = 7.f;

template <typename T>
constexpr uint32_t kAbFormat = 0;  // fields of A and B format that idesc_bf16_f32 sets and T clears
template <>
constexpr uint32_t kAbFormat<__half> = (1u << 7) | (1u << 10);
template <typename T>
__host__ __device__ constexpr uint32_t idesc(bool b_mn_major) {
  return idesc_bf16_f32(128, 128, false, b_mn_major) & ~kAbFormat<T>;
}

// Warp-uniform wait; what follows the first test is a call, one copy of it.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const PagedAttnArgs& a, int where) {
  const bool ok = paged_wait(bar, parity, a.status, a.wait_limit_ns, where);
  return __all_sync(0xFFFFFFFFu, ok);
}
__device__ __forceinline__ bool waitw(uint64_t* bar, uint32_t parity, const PagedAttnArgs& a, int where) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, a, where);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// ------------------------------------------------------------------ items
// Keys that all of the tokens [i0, i1) of a request attend (some of them: the
// intersection first interval by first, second by second).  Bounds move with
// the position in one direction (see hull), so the outer rows decide, with
// two exceptions that are looked at as well: GLOBAL_SLIDING's first row past
// the global ones, and CAUSAL_BLOCKWISE's last row before the last block.
__device__ __noinline__ Span common(const PagedAttnArgs& a, int q_len, int k_len, int i0, int i1) {
  int mid = i0;
  const int shift = k_len - q_len;
  if (a.mask.kind == kGlobalSliding) mid = a.mask.ng - shift;
  if (a.mask.kind == kCausalBlockwise) mid = (k_len - 1) / a.mask.block * a.mask.block - 1 - shift;
  Span c{0, 0x7FFFFFFF, 0, 0x7FFFFFFF};
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    Span s = paged_span(a, q_len, k_len, k == 0 ? i0 : k == 1 ? min(max(mid, i0), i1 - 1) : i1 - 1);
    if (s.a1 >= s.b1) s.a1 = s.a0, s.b1 = s.b0;  // one interval counts as both
    c.a0 = max(c.a0, s.a0);
    c.b0 = min(c.b0, s.b0);
    c.a1 = max(c.a1, s.a1);
    c.b1 = min(c.b1, s.b1);
  }
  return c;
}

// Key tiles of a hull: n0 from t0 on, then n1 from t1 on.
struct Tiles {
  int t0, n0, t1, n1;
};
__device__ __forceinline__ Tiles tiles_of(const Span& h) {
  Tiles u;
  u.t0 = h.a0 / kTile;
  u.n0 = h.b0 > h.a0 ? (h.b0 + kTile - 1) / kTile - u.t0 : 0;
  u.t1 = max(h.a1 / kTile, u.n0 > 0 ? u.t0 + u.n0 : 0);
  u.n1 = h.b1 > h.a1 ? max((h.b1 + kTile - 1) / kTile - u.t1, 0) : 0;
  return u;
}

// Row blocks (two sub-tiles) of request i; none when the other kernel serves it.
__device__ __forceinline__ int row_blocks(const PagedAttnArgs& a, int q_len) {
  return few_rows(a, q_len) ? 0 : (q_len + 2 * a.tpt - 1) / (2 * a.tpt);
}

// Sums over the requests and their row blocks: block0[i] = row blocks of the
// requests before i, line[b] = key tiles of the row blocks before b (one head;
// at least one per block, so that rows without keys are written) and
// kItemCost more for each block.
__device__ void place_items(const PagedAttnArgs& a) {
  __shared__ long long part[32];
  const int tid = threadIdx.x;
  long long at = 0;
  for (int base = 0; base < a.n_seq; base += 1024) {
    const int i = base + tid;
    const long long n = i < a.n_seq ? row_blocks(a, paged_seg(a, i).q_len) : 0;
    long long total;
    const long long inc = block_scan(n, part, total);
    // rows that overlap (a bad q_start) can make more blocks than there is room for
    if (i < a.n_seq) a.block0[i] = static_cast<int>(min(at + inc - n, static_cast<long long>(a.max_blocks)));
    at += total;
  }
  const int blocks = static_cast<int>(min(at, static_cast<long long>(a.max_blocks)));
  if (tid == 0) a.block0[a.n_seq] = blocks;
  __syncthreads();
  at = 0;
  for (int base = 0; base < blocks; base += 1024) {
    const int b = base + tid;
    long long n = 0;
    if (b < blocks) {
      int i = 0;  // the last request whose blocks start at or before b
      for (int hi = a.n_seq; hi - i > 1;) {
        const int mid = (i + hi) >> 1;
        if (a.block0[mid] <= b) i = mid; else hi = mid;
      }
      const SegInfo sg = paged_seg(a, i);
      const int tok = (b - a.block0[i]) * 2 * a.tpt;
      if (tok < sg.q_len) {
        const Tiles t = tiles_of(hull(a, sg.q_len, sg.k_len, tok, min(tok + 2 * a.tpt, sg.q_len)));
        n = max(t.n0 + t.n1, 1) + kItemCost;
      }
    }
    long long total;
    const long long inc = block_scan(n, part, total);
    if (b < blocks) a.line[b] = at + inc - n;
    at += total;
  }
  if (tid == 0) a.line[blocks] = at;
}

// First kernel of a call: clears the status and the counts, reports lengths
// that the tensors do not hold, and places the items of many rows.
__global__ void __launch_bounds__(1024) paged_begin_kernel(const __grid_constant__ PagedAttnArgs a, bool many) {
  launch_dependents();
  for (int i = threadIdx.x; i <= kPagedMaxSpans; i += 1024) a.arrived[i] = 0;  // and the claims behind them
  if (many && threadIdx.x < kPagedMaxChunkCtas) a.cuts[threadIdx.x].last = -1;
  if (threadIdx.x < 4) a.status[threadIdx.x] = 0;
  __syncthreads();
  const int room = a.max_pages * a.page_size;
  for (int i = threadIdx.x; i < a.n_seq; i += 1024) {
    const int r0 = a.q_start[i], r1 = a.q_start[i + 1], kl = a.k_len[i];
    if (r0 < 0 || r1 < r0 || r1 > a.Tq || kl < 0 || kl > room) paged_report(a.status, kStatusDeviceArg, 50);
    if (a.ctx_len) {
      const int c = a.ctx_len[i];
      if (c < 0 || c > room || paged_seg(a, i).q_len < paged_rows(a, i).q_len)
        paged_report(a.status, kStatusDeviceArg, 52);
    }
  }
  if (many) place_items(a);
}

// The line of tiles: request by request, head by head, block by block.  An
// item's kItemCost come before its tiles; a span that ends within them has
// no piece of it.
struct Line {
  long long total, ctas;
  __device__ __forceinline__ Line(const PagedAttnArgs& a, int grid) {
    // requests whose rows do not overlap make fewer than 2^52 places; a q_start
    // that lets them overlap may make more, and is reported and not served then
    const long long head = a.line[a.block0[a.n_seq]];
    total = head < (1LL << 52) / a.Hkv ? head * a.Hkv : 0;
    ctas = min(static_cast<long long>(grid), max(total / kMinTiles, 1LL));
  }
  __device__ __forceinline__ long long start(long long c) const { return line_div(min(c, ctas) * total, ctas); }
  __device__ __forceinline__ long long cta_of(long long p) const {
    return line_div((p + 1) * ctas - 1, total);
  }
};

struct Place {
  int seq, head, block;  // block: inside the request
  long long first;       // of the item's tiles on the line
  int tiles;
};
__device__ __noinline__ Place locate(const PagedAttnArgs& a, long long pos) {
  int lo = 0, hi = a.n_seq;  // the last request that starts at or before pos
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.line[a.block0[mid]] * a.Hkv <= pos) lo = mid; else hi = mid;
  }
  Place p;
  p.seq = lo;
  const int b0 = a.block0[lo], b1 = a.block0[lo + 1];
  const long long l0 = a.line[b0], per = a.line[b1] - l0;  // tiles of one head
  const long long rel = pos - l0 * a.Hkv;
  p.head = static_cast<int>(line_div(rel, per));
  const long long in = rel - p.head * per + l0;
  lo = b0, hi = b1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.line[mid] <= in) lo = mid; else hi = mid;
  }
  p.block = lo - b0;
  p.first = pos - (in - a.line[lo]) + kItemCost;
  p.tiles = static_cast<int>(a.line[lo + 1] - a.line[lo]) - kItemCost;
  return p;
}

// Slot of CTA c's sums of the item whose tiles start at `first`: 2 c when it
// is the first piece of its span, 2 c + 1 for a later one.
__device__ __forceinline__ long long slot_of(const Line& ln, long long c, long long first) {
  return 2 * c + (ln.start(c) < first - kItemCost ? 1 : 0);
}

// ------------------------------------------------------------------ scheduler
__device__ __forceinline__ void scheduler(const PagedAttnArgs& a, const Line& ln, uint64_t* bar, Item* items) {
  const int lane = threadIdx.x & 31;
  long long pos = ln.start(blockIdx.x);
  const long long end = ln.start(blockIdx.x + 1);
  Place p{};
  SegInfo sg{};
  int b0 = 0, b1 = 0;  // the request's row blocks
  bool begun = false;
  for (int it = 0;;) {
    const int slot = it % kItemSlots;
    if (pos >= end) {
      if (it >= kItemSlots && !waitw(&bar[B_ITEMPTY + slot], (it / kItemSlots - 1) & 1, a, 60)) return;
      if (lane == 0) {
        items[slot].valid = 0;
        mbar_arrive(&bar[B_ITFULL + slot]);
      }
      return;
    }
    if (!begun) {
      begun = true;
      p = locate(a, pos);
      sg = paged_seg(a, p.seq);
      b0 = a.block0[p.seq];
      b1 = a.block0[p.seq + 1];
    } else {  // the next block, head or request
      p.first = pos + kItemCost;
      if (++p.block == b1 - b0) {
        p.block = 0;
        if (++p.head == a.Hkv) {
          p.head = 0;
          if (p.seq + 1 >= a.n_seq) {  // only if the lengths changed meanwhile
            pos = end;
            continue;
          }
          do {
            ++p.seq;
            b0 = b1;
            b1 = a.block0[p.seq + 1];
          } while (b1 == b0 && p.seq + 1 < a.n_seq);
          sg = paged_seg(a, p.seq);
        }
      }
      p.tiles = static_cast<int>(a.line[b0 + p.block + 1] - a.line[b0 + p.block]) - kItemCost;
    }
    const long long from = max(pos, p.first), to = min(p.first + p.tiles, end);
    pos = min(p.first + p.tiles, end);
    if (from >= to) continue;
    const int tok0 = p.block * 2 * a.tpt, toks = min(2 * a.tpt, sg.q_len - tok0);
    const bool narrow = toks <= a.tpt;
    const int u0 = static_cast<int>(from - p.first), take = static_cast<int>(to - from);
    // lanes 0 and 1: a sub-tile's ranges; the others the item's
    const int x = lane < 2 && !narrow ? lane : 0;
    const int i0 = tok0 + (lane < 2 ? x * a.tpt : 0), i1 = lane < 2 ? min(i0 + a.tpt, sg.q_len) : tok0 + toks;
    const Span h = hull(a, sg.q_len, sg.k_len, i0, i1), f = common(a, sg.q_len, sg.k_len, i0, i1);
    if (it >= kItemSlots && !waitw(&bar[B_ITEMPTY + slot], (it / kItemSlots - 1) & 1, a, 60)) return;
    Item& inf = items[slot];
    if (lane < 2) {
      inf.hull[lane] = h;
      inf.full[lane] = f;
    } else if (lane == 2) {
      const Tiles tl = tiles_of(h);
      inf.all = h;
      inf.every = f;
      inf.valid = 1;
      inf.narrow = narrow;
      inf.n = tl.n0 + tl.n1 > 0 ? take : 0;
      inf.u0 = u0;
      inf.head = p.head;
      inf.tok0 = tok0;
      inf.part = take < p.tiles ? static_cast<int>(slot_of(ln, blockIdx.x, p.first)) : -1;
      inf.seq = p.seq;
      inf.q_off = sg.q_off;
      inf.q_len = sg.q_len;
      inf.k_len = sg.k_len;
      inf.t0 = tl.t0;
      inf.n0 = tl.n0;
      inf.t1 = tl.t1;
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bar[B_ITFULL + slot]);
      // an item that starts here and goes on in later spans, for the join
      if (u0 == 0 && take < p.tiles)
        a.cuts[blockIdx.x] = PagedCut{static_cast<int>(ln.cta_of(p.first + p.tiles - 1)),
                                      static_cast<int>(slot_of(ln, blockIdx.x, p.first) & 1),
                                      p.head,
                                      tok0,
                                      sg.q_off,
                                      sg.q_len,
                                      {0, 0}};
    }
    ++it;
  }
}

// ------------------------------------------------------------------ producer
__device__ __forceinline__ void producer(const PagedAttnArgs& a, const CUtensorMap* tq, const CUtensorMap* tk,
                                         const CUtensorMap* tv, uint8_t* sQ, uint8_t* sKV, uint64_t* bar,
                                         const Item* items) {
  const int lane = threadIdx.x & 31;
  const int boxes = kTile / a.box_rows;  // per tile and half
  const int box = lane % boxes, half = lane / boxes;
  const uint32_t q_bytes = static_cast<uint32_t>(a.tpt * a.G) * 128;  // of one 64-value half of a sub-tile
  uint32_t kv_iter = 0, issued = 0;
  int q_issued = 0;
  for (int it = 0;; ++it) {
    const int slot = it % kItemSlots;
    if (!waitw(&bar[B_ITFULL + slot], (it / kItemSlots) & 1, a, 61)) break;
    const Item inf = items[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_ITEMPTY + slot]);
    if (!inf.valid) return;
    if (it >= 1 && !waitw(&bar[B_QEMPTY], (it - 1) & 1, a, 63)) break;
    if (lane == 0) {
      const int subs = inf.narrow ? 1 : 2;
      mbar_arrive_expect_tx(&bar[B_QFULL], 2 * subs * q_bytes);
      for (int x = 0; x < subs; ++x)
        for (int c = 0; c < 2; ++c)
          tma_load_3d(sQ + x * kTileBytes + c * kChunkBytes, tq, &bar[B_QFULL], c * 64, inf.head * a.G,
                      inf.q_off + inf.tok0 + x * a.tpt);
    }
    q_issued = it + 1;

    const int* table = a.table + inf.seq * a.table_stride;
    // page of this lane's box of tile t (n_pages, past the array, where none is
    // needed or the entry is no page: that box is filled with zeros)
    auto entry = [&](int t) -> int {
      const int j = inf.tile(t) * kTile + box * a.box_rows;
      if (!span_hits(inf.all, j, j + a.box_rows)) return a.n_pages;
      const int pg = __ldg(table + j / a.page_size);
      if (pg < 0 || pg >= a.n_pages) {
        paged_report(a.status, kStatusDeviceArg, 51);
        return a.n_pages;
      }
      return pg;
    };
    int next = inf.n > 0 ? entry(0) : 0;
    bool ok = true;
    for (int t = 0; t < inf.n && ok; ++t) {
      const int page = next;
      const int y = (inf.tile(t) * kTile + box * a.box_rows) % a.page_size;
      if (t + 1 < inf.n) next = entry(t + 1);
#pragma unroll
      for (int which = 0; which < 2; ++which) {  // K(t) then V(t)
        const uint32_t idx = kv_iter + 2 * t + which;
        const int stg = idx % kStages;
        if (idx >= kStages && !waitw(&bar[B_KVEMPTY + stg], ((idx / kStages) - 1) & 1, a, 62)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bar[B_KVFULL + stg], kTileBytes);
        __syncwarp();
        if (half < 2)
          tma_load_4d(sKV + stg * kTileBytes + half * kChunkBytes + box * a.box_rows * 128, which ? tv : tk,
                      &bar[B_KVFULL + stg], half * 64, a.head_first ? inf.head : y, a.head_first ? y : inf.head, page);
        issued = idx + 1;
      }
    }
    if (!ok) break;
    kv_iter += 2 * inf.n;
  }
  // a wait ran out: let the copies already issued land before the CTA leaves
  for (uint32_t d = 0; d < kStages && d < issued; ++d) {
    const uint32_t idx = issued - 1 - d;
    mbar_wait(&bar[B_KVFULL + idx % kStages], (idx / kStages) & 1, nullptr, 100000000ull, 0, 0);
  }
  if (q_issued >= 1) mbar_wait(&bar[B_QFULL], (q_issued - 1) & 1, nullptr, 100000000ull, 0, 0);
}

// ------------------------------------------------------------------ MMA issuer
template <typename T>
__device__ __forceinline__ void mma_issuer(const PagedAttnArgs& a, uint8_t* sQ, uint8_t* sKV, uint64_t* bar,
                                           const Item* items, uint32_t tbase) {
  constexpr uint32_t kIdescS = idesc<T>(false);  // S = Q K^T (both K-major)
  constexpr uint32_t kIdescO = idesc<T>(true);   // O += P V (P in TMEM, V N-major)
  const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
  const uint64_t dK0 = sdesc_sw128(smem_u32(sKV), 16, 1024);
  const uint64_t dV0 = sdesc_sw128(smem_u32(sKV), kChunkBytes, 1024);
  uint32_t kv_iter = 0;
  uint32_t p_iss[3] = {0, 0, 0};
  auto scores = [&](int buf, int sub, int kst, int full) {
    const uint64_t dK = desc_add(dK0, kst * kTileBytes), dQ = desc_add(dQ0, sub * kTileBytes);
    tc_fence_after();
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t off = (ks >> 2) * kChunkBytes + (ks & 3) * 32;
      umma_ss(tbase + 128 * buf, desc_add(dQ, off), desc_add(dK, off), kIdescS, ks > 0 ? 1u : 0u);
    }
    umma_commit(&bar[B_SFULL + full]);
  };
  auto values = [&](int buf, int sub, int vst, bool first) {
    const uint64_t dV = desc_add(dV0, vst * kTileBytes);
    tc_fence_after();
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      umma_ts(tbase + 256 + 128 * sub, tbase + 128 * buf + 8 * ks, desc_add(dV, ks * 2048), kIdescO,
              ks > 0 || !first ? 1u : 0u);
    umma_commit(&bar[B_OFULL + sub]);
  };
  for (int it = 0;; ++it) {
    const int slot = it % kItemSlots;
    if (!waitw(&bar[B_ITFULL + slot], (it / kItemSlots) & 1, a, 70)) goto abort;
    {
      const Item& inf = items[slot];
      if (!inf.valid) return;
      const int n = inf.n;
      if (!waitw(&bar[B_QFULL], it & 1, a, 71)) goto abort;
      auto kv_full = [&](uint32_t idx) { return waitw(&bar[B_KVFULL + idx % kStages], (idx / kStages) & 1, a, 72); };
      if (inf.narrow) {
        // S(0), S(1), PV(0), S(2), PV(1), ...: tile t in score buffer t & 1
        for (int t = 0; t <= n; ++t) {
          if (t < n) {
            const uint32_t kidx = kv_iter + 2 * t;
            if (!kv_full(kidx)) goto abort;
            scores(t & 1, 0, kidx % kStages, (t & 1) ? 2 : 0);
            umma_commit(&bar[B_KVEMPTY + kidx % kStages]);
            if (t == n - 1) umma_commit(&bar[B_QEMPTY]);
          }
          if (t >= 1) {
            const uint32_t vidx = kv_iter + 2 * (t - 1) + 1;
            const int odd = (t - 1) & 1, full = odd ? 2 : 0;
            if (!kv_full(vidx)) goto abort;
            if (!waitw(&bar[B_PFULL + full], (odd ? p_iss[2] : p_iss[0]) & 1, a, 73)) goto abort;
            if (odd) ++p_iss[2]; else ++p_iss[0];
            values(odd, 0, vidx % kStages, t == 1);
            umma_commit(&bar[B_KVEMPTY + vidx % kStages]);
          }
        }
      } else {
        bool first[2] = {true, true};
        uint32_t prev[2] = {kTileEmpty, kTileEmpty};
        for (int t = 0; t <= n; ++t) {
          const uint32_t vidx = kv_iter + 2 * (t - 1) + 1, kidx = kv_iter + 2 * t;
          const int kt = t < n ? inf.tile(t) : 0;
          bool v_ready = false, k_ready = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (prev[x] != kTileEmpty) {  // O_x += P_x(t-1) V(t-1), before S_x(t) overwrites P_x
              if (!v_ready && !kv_full(vidx)) goto abort;
              v_ready = true;
              if (!waitw(&bar[B_PFULL + x], p_iss[x] & 1, a, 74)) goto abort;
              ++p_iss[x];
              values(x, x, vidx % kStages, first[x]);
              first[x] = false;
            }
            prev[x] = t < n ? inf.cls(x, kt) : kTileEmpty;
            if (prev[x] != kTileEmpty) {
              if (!k_ready && !kv_full(kidx)) goto abort;
              k_ready = true;
              scores(x, x, kidx % kStages, x);
            }
          }
          if (t >= 1) {
            if (!v_ready && !kv_full(vidx)) goto abort;  // released only once it has landed
            umma_commit(&bar[B_KVEMPTY + vidx % kStages]);
          }
          if (t < n) {
            if (!k_ready && !kv_full(kidx)) goto abort;
            umma_commit(&bar[B_KVEMPTY + kidx % kStages]);
            if (t == n - 1) umma_commit(&bar[B_QEMPTY]);
          }
        }
      }
      if (n == 0) umma_commit(&bar[B_QEMPTY]);
      kv_iter += 2 * n;
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bar[B_ITEMPTY + slot]);
    }
  }
abort:
  umma_commit(&bar[B_DRAIN]);
  mbar_wait(&bar[B_DRAIN], 0, nullptr, 100000000ull, 0, 0);
}

// ------------------------------------------------------------------ softmax warpgroup
// A partly masked tile: -inf over the scores whose bit is clear, in TMEM, so
// that one copy of what follows serves every tile.
__device__ __forceinline__ void mask_scores(uint32_t tS, const Span& sp, int j0) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const uint32_t bits = span_bits(sp, j0 + 32 * c);
    uint32_t r[32];
    tmem_ld32(tS + 32 * c, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = ((bits >> k) & 1u) ? r[k] : 0xFF800000u;
    tmem_st32(tS + 32 * c, r);
  }
  tmem_st_wait();
}

// Maximum of the thread's 128 scores, 64 columns at a time: eight independent
// partial maxima, so that the row is not one dependency chain.
__device__ __forceinline__ float row_max(uint32_t tS) {
  float mp[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mp[j] = -INFINITY;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r0[32], r1[32];
    tmem_ld32(tS + 64 * h, r0);
    tmem_ld32(tS + 64 * h + 32, r1);
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mp[j] = fmax3(mp[j], __uint_as_float(r0[16 * g + j]), __uint_as_float(r0[16 * g + 8 + j]));
        mp[j] = fmax3(mp[j], __uint_as_float(r1[16 * g + j]), __uint_as_float(r1[16 * g + 8 + j]));
      }
  }
  return fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
}

// p = 2^(s scale log2(e) - base) of 32 columns, written as pairs over the
// columns of S read before; the next 32 are requested meanwhile.
template <typename T>
__device__ __forceinline__ void exp_chunk(uint32_t tS, int c, const uint32_t (&cur)[32], uint32_t (&nxt)[32],
                                          uint64_t sl2x2, uint64_t nb2, uint64_t (&acc)[4]) {
  tmem_ld_wait();
  if (c + 1 < 4) tmem_ld32(tS + 32 * (c + 1), nxt);
  uint32_t pk[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint64_t xx = ffma2(f2(__uint_as_float(cur[2 * k]), __uint_as_float(cur[2 * k + 1])), sl2x2, nb2);
    const uint64_t pp = f2(ex2_approx(f2lo(xx)), ex2_approx(f2hi(xx)));
    acc[k & 3] = fadd2(acc[k & 3], pp);
    pk[k] = Half2<T>::pack(f2lo(pp), f2hi(pp));
  }
  tmem_st16(tS + 16 * c, pk);
}
template <typename T>
__device__ __forceinline__ float row_exp(uint32_t tS, float sl2, float base) {
  const uint64_t sl2x2 = f2(sl2, sl2), nb2 = f2(-base, -base);
  uint64_t acc[4] = {0, 0, 0, 0};
  uint32_t ra[32], rb[32];
  tmem_ld32(tS, ra);
#pragma unroll
  for (int c = 0; c < 4; c += 2) {
    exp_chunk<T>(tS, c, ra, rb, sl2x2, nb2, acc);
    exp_chunk<T>(tS, c + 1, rb, ra, sl2x2, nb2, acc);
  }
  const uint64_t t = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
  return f2lo(t) + f2hi(t);
}

// Values that are not finite in keys that only some rows of an item attend
// must not meet a p of 0.  Before a tile's product they are set to zero in
// shared memory, value by value, by each warpgroup that has a product with the
// tile (both write the same); at the end the rows that attend such a key add
// the values to their sums.  A weight is positive, so whatever it is, its
// product with an infinity or NaN is that same value, and no score is needed
// for it.  In a key that all rows of the item attend the value stays in the
// product, where an infinity becomes NaN if the row's weight has rounded to 0:
// not finite either way, and a scan of every tile is saved.
//
// One such value in a chunk of 256 tokens at 131K keys takes the call from 0.82
// to 0.90 ms; what all calls pay for it is a look at the keys of partial tiles
// and more code (8 prompts 278 -> 284 us).
//
// Row `key` of the V tile (one thread per key): whether it holds such a value,
template <typename T>
__device__ __forceinline__ bool bad_v_row(const uint8_t* v, int key) {
  uint32_t bad = 0;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(v + (i >> 3) * kChunkBytes + key * 128 + (((i ^ key) & 7) << 4));
    bad |= Half2<T>::not_finite(w.x) | Half2<T>::not_finite(w.y) | Half2<T>::not_finite(w.z) | Half2<T>::not_finite(w.w);
  }
  return (bad & 0x80008000u) != 0;
}
// and its values without them,
template <typename T>
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  return w & ~(((Half2<T>::not_finite(w) & 0x80008000u) >> 15) * 0xFFFFu);
}
template <typename T>
__device__ __noinline__ void finite_v_row(uint8_t* v, int key) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    uint4* at = reinterpret_cast<uint4*>(v + (i >> 3) * kChunkBytes + key * 128 + (((i ^ key) & 7) << 4));
    const uint4 w = *at;
    *at = make_uint4(finite_part<T>(w.x), finite_part<T>(w.y), finite_part<T>(w.z), finite_part<T>(w.w));
  }
}
// or none at all (no row of the item attends the key, and nothing of
// what lies there may reach a result).
__device__ __forceinline__ void clear_v_row(uint8_t* v, int key) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    *reinterpret_cast<uint4*>(v + (i >> 3) * kChunkBytes + key * 128 + (((i ^ key) & 7) << 4)) = make_uint4(0, 0, 0, 0);
}

// Writes a warp's rows, one per lane, of an item that had such values, adding
// them from the cache; all lanes take part.  tO: the products' sums.
template <typename T>
__device__ __noinline__ void write_hidden(const PagedAttnArgs& a, const Item& inf, int x, uint32_t tO, bool valid,
                                          Span sp, T* orow, float* part, float l) {
  const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
  const int* table = a.table + inf.seq * a.table_stride;
  const T* v = static_cast<const T*>(a.vc) + inf.head * a.head_stride;
  // place of key j's values in v, -1 where all rows or none attend it or it has no page
  auto place = [&](int j) -> long long {
    if (!in_span(inf.all, j) || in_span(inf.every, j)) return -1;
    const int page = __ldg(table + j / a.page_size);
    return page < 0 || page >= a.n_pages ? -1 : page * a.page_stride + j % a.page_size * a.token_stride;
  };
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    __syncwarp();
    tmem_ld32(tO + 32 * c, r);
    tmem_ld_wait();
#pragma unroll 1
    for (int t = 0; t < inf.n; ++t) {
      const int kt = inf.tile(t);
      if (span_covers(inf.every, kt * kTile, kt * kTile + kTile) || (!inf.narrow && inf.cls(x, kt) == kTileEmpty))
        continue;
#pragma unroll 1
      for (int j0 = kt * kTile; j0 < (kt + 1) * kTile; j0 += 32) {
        const long long at = place(j0 + (threadIdx.x & 31));
        uint32_t bad = 0;
        if (at >= 0)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 w = *reinterpret_cast<const uint4*>(v + at + 32 * c + 8 * u);
            bad |= Half2<T>::not_finite(w.x) | Half2<T>::not_finite(w.y) | Half2<T>::not_finite(w.z) |
                   Half2<T>::not_finite(w.w);
          }
        for (uint32_t keys = __ballot_sync(0xFFFFFFFFu, bad & 0x80008000u); keys != 0; keys &= keys - 1) {
          const int j = __ffs(keys) - 1;
          const T* vj = v + __shfl_sync(0xFFFFFFFFu, at, j) + 32 * c;
          if (!in_span(sp, j0 + j)) continue;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(vj + 2 * u);
            const float2 f = Half2<T>::unpack(w ^ finite_part<T>(w));  // zero where it is finite
            r[2 * u] = __float_as_uint(__uint_as_float(r[2 * u]) + f.x);
            r[2 * u + 1] = __float_as_uint(__uint_as_float(r[2 * u + 1]) + f.y);
          }
        }
      }
    }
    if (!valid) continue;
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float y0 = __uint_as_float(r[k]) * inv, y1 = __uint_as_float(r[k + 1]) * inv;
      if (part)
        *reinterpret_cast<float2*>(part + 32 * c + k) = make_float2(y0, y1);
      else
        *reinterpret_cast<uint32_t*>(orow + 32 * c + k) = Half2<T>::pack(y0, y1);
    }
  }
}

template <typename T>
__device__ __forceinline__ void softmax_wg(const PagedAttnArgs& a, int x, uint64_t* bar, const Item* items,
                                           uint8_t* sKV, volatile int* hidden, uint32_t tbase) {
  const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = wq * 32 + lane;  // TMEM lane = row of the sub-tile
  const uint32_t tl = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t tO = tbase + tl + 256 + 128 * x;
  const float sl2 = a.scale_log2;
  uint32_t s_cnt = 0, s_odd = 0;  // phases of the score barriers so far
  uint32_t o_cnt = 0;          // products into this sub-tile's O so far
  uint32_t kv_iter = 0;
  for (int it = 0;; ++it) {
    const int slot = it % kItemSlots;
    if (!waitw(&bar[B_ITFULL + slot], (it / kItemSlots) & 1, a, 80 + x)) return;
    const Item& inf = items[slot];
    if (!inf.valid) return;
    const bool narrow = inf.narrow != 0;
    const int n = inf.n;
    if (narrow && x == 1) {  // the other warpgroup's item
      kv_iter += 2 * n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_ITEMPTY + slot]);
      continue;
    }
    const int tok_in = row / a.G;
    const int token = inf.tok0 + x * a.tpt + tok_in;
    const int head = inf.head * a.G + row - tok_in * a.G;
    const bool valid = tok_in < a.tpt && token < inf.q_len;
    const Span sp = paged_span(a, inf.q_len, inf.k_len, min(token, inf.q_len - 1));
    float m = -INFINITY, l = 0.f;
    bool any = false;
    for (int t = 0; t < n; ++t) {
      const int kt = inf.tile(t);
      const uint32_t cls = inf.cls(x, kt);
      if (!narrow && cls == kTileEmpty) continue;
      const bool odd = narrow && (t & 1);  // an odd tile of a narrow item
      const int buf = odd ? 1 : x, full = odd ? 2 : x;
      const uint32_t tS = tbase + tl + 128 * buf;
      if (!waitw(&bar[B_SFULL + full], (odd ? s_odd : s_cnt) & 1, a, 82 + x)) return;
      if (odd) ++s_odd; else ++s_cnt;
      tc_fence_after();
      if (!span_covers(inf.every, kt * kTile, kt * kTile + kTile)) {
        // only now: a warpgroup that skipped a narrow item runs ahead of the
        // loads, and the scores show that the ring has come to this tile
        const uint32_t vidx = kv_iter + 2 * t + 1;
        if (!waitw(&bar[B_KVFULL + vidx % kStages], (vidx / kStages) & 1, a, 88 + x)) return;
        const int j = kt * kTile + row;
        uint8_t* v = sKV + (vidx % kStages) * kTileBytes;
        if (!in_span(inf.all, j)) {
          clear_v_row(v, row);
        } else if (!in_span(inf.every, j) && bad_v_row<T>(v, row)) {
          // the other warpgroup may find the value gone, but then the mark set
          hidden[slot] = it + 1;
          __threadfence_block();
          finite_v_row<T>(v, row);
        }
        fence_proxy_async_smem();
        if (cls != kTileFull) mask_scores(tS, sp, kt * kTile);
      }
      const float mx = row_max(tS);
      const float m_new = fmaxf(m, mx * sl2);
      float factor = 1.f;
      bool need = false;
      if (!any) {
        m = m_new;
      } else if (m_new > m + kRescaleThreshold) {
        factor = ex2_approx(m - m_new);
        need = true;
        m = m_new;
      }
      const float base = (m == -INFINITY ? 0.f : m) - kBias<T>;
      const float sum = row_exp<T>(tS, sl2, base);
      l = l * factor + sum;
      const bool rescale = __any_sync(0xFFFFFFFFu, need);
      // The product before this one must have finished before O is rescaled.
      // In a narrow item nothing else tells that it has (the next scores do
      // not come after it), and it must be known before another one starts: a
      // wait by parity cannot tell the last phase from the last but two.
      if (any && (rescale || narrow)) {
        if (!waitw(&bar[B_OFULL + x], (o_cnt - 1) & 1, a, 84 + x)) return;
        tc_fence_after();
      }
      if (rescale) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * factor);
          tmem_st32(tO + 32 * c, r);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_PFULL + full]);
      ++o_cnt;
      any = true;
    }
    kv_iter += 2 * n;
    if (any) {
      if (!waitw(&bar[B_OFULL + x], (o_cnt - 1) & 1, a, 86 + x)) return;
      tc_fence_after();
    }
    T* orow = static_cast<T*>(a.o) + (static_cast<long long>(inf.q_off + (valid ? token : 0)) * a.Hq + head) * kHeadDim;
    float* part = inf.part < 0 ? nullptr : a.chunk_parts + inf.part * static_cast<long long>(kPagedChunkPartFloats);
    // the other warpgroup may set the mark just now, for tiles of its own alone:
    // a vote, since what follows takes all lanes of the warp together
    if (__any_sync(0xFFFFFFFFu, any && hidden[slot] == it + 1)) {
      write_hidden<T>(a, inf, x, tO, valid, sp, orow, part ? part + (x * 128 + row) * kHeadDim : nullptr, l);
    } else if (any) {
      const float inv = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
      if (part) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + 32 * c, r);
          tmem_ld_wait();
          if (valid) {
            float* dst = part + (x * 128 + row) * kHeadDim + 32 * c;
#pragma unroll
            for (int u = 0; u < 4; ++u) st_global_v8(dst + 8 * u, &r[8 * u]);
          }
        }
      } else {
        // Four lanes exchange 32-byte pieces of their rows, so that a store
        // covers 8 lines of 128 bytes and not 32 pieces of 32: 32 requests of
        // 5 tokens 165.1 -> 162.3 us; prompts are the same either way.
        const int place = valid ? static_cast<int>((orow - static_cast<T*>(a.o)) / kHeadDim) : -1, quad = lane & 3;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
            tmem_ld32(tO + 64 * h + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[16 * c + k] = Half2<T>::pack(__uint_as_float(r[2 * k]) * inv, __uint_as_float(r[2 * k + 1]) * inv);
          }
#pragma unroll
          for (int d = 1; d <= 2; d <<= 1)
#pragma unroll
            for (int p = 0; p < 4; ++p)
              if (!(p & d))
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  uint32_t &lo = w[8 * p + e], &hi = w[8 * (p + d) + e];
                  const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, (quad & d) ? lo : hi, d);
                  if (quad & d) lo = got; else hi = got;
                }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // now piece `quad` of the quad's row k
            const int at = __shfl_sync(0xFFFFFFFFu, place, (lane & ~3) + k);
            if (at < 0) continue;
            T* dst = static_cast<T*>(a.o) + static_cast<long long>(at) * kHeadDim + 64 * h + 16 * quad;
            if (a.out_v8) {
              st_global_v8(dst, &w[8 * k]);
            } else {
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[8 * k], w[8 * k + 1], w[8 * k + 2], w[8 * k + 3]);
              *reinterpret_cast<uint4*>(dst + 8) =
                  make_uint4(w[8 * k + 4], w[8 * k + 5], w[8 * k + 6], w[8 * k + 7]);
            }
          }
        }
      }
    } else if (valid && !part) {
#pragma unroll
      for (int u = 0; u < 16; ++u) *reinterpret_cast<uint4*>(orow + 8 * u) = make_uint4(0, 0, 0, 0);
    }
    if (valid && part) {
      part[256 * kHeadDim + x * 128 + row] = m;
      part[256 * kHeadDim + 256 + x * 128 + row] = any ? l : 0.f;
    } else if (valid) {
      a.lse[static_cast<long long>(head) * a.Tq + inf.q_off + token] =
          !any || l == 0.f ? -INFINITY : (m + log2f(l) - kBias<T>) * kLn2;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_ITEMPTY + slot]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm + kOffQ;
  uint8_t* sKV = sm + kOffKV;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + kOffCtl);
  Item* items = reinterpret_cast<Item*>(sm + kOffCtl + 256);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kOffCtl + 896);
  // per item slot: the last item (from 1) with values that write_hidden adds;
  // a warp may be that many items ahead of another
  int* hidden = reinterpret_cast<int*>(sm + kOffCtl + 904);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int b = 0; b < B_COUNT; ++b) mbar_init(&bar[b], 1);
    for (int x = 0; x < 3; ++x) mbar_init(&bar[B_PFULL + x], 4);  // one arrival per softmax warp
    for (int x = 0; x < kItemSlots; ++x) hidden[x] = 0;
    for (int x = 0; x < kItemSlots; ++x) mbar_init(&bar[B_ITEMPTY + x], 10);  // softmax, MMA and producer warps
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  grid_wait();          // the items have their places on the line
  launch_dependents();  // and what follows this kernel need not wait for the one before it
  const Line ln(a, gridDim.x);
  // a CTA without a span finds no item
  if (warp == 10)
    scheduler(a, ln, bar, items);
  else if (warp == 9)
    producer(a, &tmQ, &tmK, &tmV, sQ, sKV, bar, items);
  else if (warp == 8)
    mma_issuer<T>(a, sQ, sKV, bar, items, tbase);
  else
    softmax_wg<T>(a, warp >> 2, bar, items, sKV, hidden, tbase);
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the pieces of the item that starts in CTA blockIdx.x's span and ends
// in a later one's: 32 rows per block, four rows per warp.  Bound by trips to
// L2, so the loads of two pieces of all four rows are under way at once; launched
// alone and cold 6.5 us for 32 requests of 5 tokens, 10.9 for 8 prompts.
constexpr int kJoinRows = 32;
template <typename T>
__global__ void __launch_bounds__(8 * kJoinRows, 3) paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  launch_dependents();
  grid_wait();
  const int c0 = blockIdx.x;
  const PagedCut cut = a.cuts[c0];
  if (cut.last < 0) return;
  const int lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kJoinRows + (threadIdx.x >> 5) * 4;  // of the item's two sub-tiles
  auto token_of = [&](int row) { return cut.tok0 + (row >> 7) * a.tpt + (row & 127) / a.G; };
  if (token_of(row0) >= cut.q_len || (row0 & 127) >= a.tpt * a.G) return;  // nor do the three after it have a token
  auto piece = [&](int k) {
    return a.chunk_parts + (2 * (c0 + k) + (k == 0 ? cut.late : 0)) * static_cast<long long>(kPagedChunkPartFloats);
  };
  float m, l, o[4][4];
  join_rows<256, 4, 2>(cut.last - c0 + 1, piece, row0, m, l, o);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float mr = __shfl_sync(~0u, m, 8 * r), lr = __shfl_sync(~0u, l, 8 * r);
    const int row = row0 + r, token = token_of(row);
    if (token >= cut.q_len || (row & 127) >= a.tpt * a.G) continue;
    const int head = cut.head * a.G + (row & 127) % a.G;
    const float inv = lr == 0.f ? 0.f : 1.f / lr;
    T* dst = static_cast<T*>(a.o) + (static_cast<long long>(cut.q_off + token) * a.Hq + head) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Half2<T>::pack(o[r][0] * inv, o[r][1] * inv), Half2<T>::pack(o[r][2] * inv, o[r][3] * inv));
    if (lane == 0)
      a.lse[static_cast<long long>(head) * a.Tq + cut.q_off + token] =
          lr == 0.f ? -INFINITY : (mr + log2f(lr) - kBias<T>) * kLn2;
  }
}

template <typename T>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                   int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(paged_chunk_kernel<T>, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_after(paged_chunk_kernel<T>, dim3(std::min(num_sms, kPagedMaxChunkCtas)), kThreads, kSmemBytes, st, tq,
                      tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_begin(const PagedAttnArgs& a, bool many, cudaStream_t st) {
  note_launches(1);
  paged_begin_kernel<<<1, 1024, 0, st>>>(a, many);
  return cudaGetLastError();
}

cudaError_t launch_paged_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch<__half>(tq, tk, tv, a, num_sms, st) : launch<__nv_bfloat16>(tq, tk, tv, a, num_sms, st);
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st) {
  const dim3 grid(std::min(num_sms, kPagedMaxChunkCtas), 256 / kJoinRows);
  note_launches(1);
  return launch_after(fp16 ? paged_join_kernel<__half> : paged_join_kernel<__nv_bfloat16>, grid, 8 * kJoinRows, 0, st,
                      a);
}

}  // namespace lca
