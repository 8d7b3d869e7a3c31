// lca_paged_api.cu — the paged-cache entry points of include/lca_attn.h:
// argument checks (all before anything is launched), workspace layout and
// launches.  Nothing here allocates or throws.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/lca_attn.h"
#include "lca_host.h"
#include "lca_paged.h"
#include "lca_paged8.h"

namespace lca {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool overlap(const void* a, long long na, const void* b, long long nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// int32 device memory that holds n values (n = 0: anything).
bool ints(const int32_t* p, long long n) { return n == 0 || (p && aligned4(p) && device_input(p)); }

constexpr long long kMaxStride = 1LL << 38;  // elements; a TMA map takes byte strides below 2^40
bool stride_ok(int64_t s) { return s >= 8 && s % 8 == 0 && s <= kMaxStride; }

// Elements from the first of n rows to the last, `stride` apart.  What is
// longer than any memory is refused before it is multiplied in 64 bits.
bool fits(long long n, int64_t stride) {
  return n <= 1 || static_cast<double>(n - 1) * static_cast<double>(stride) <= 1e15;
}
constexpr int kMostRequests = 0x3FFFFFFF;  // the kernels' loops over requests stay in 32 bits
constexpr int kMostHeads = 0xFFFFFF;       // and so do a row's elements

// A cache of either kind as the checks and launches see it: c has the values'
// layout (its dtype is of no use for an 8-bit one), c8 the factors.
struct Cache {
  const lca_paged_cache* c;
  const lca_paged_cache_fp8* c8;  // null: 16 bits
  long long bytes() const { return c8 ? 1 : 2; }
};

lca_status check_cache(const lca_paged_cache* c) {
  if (!c) return LCA_ERR_INVALID_ARG;
  if (c->dtype != LCA_BF16 && c->dtype != LCA_F16) return LCA_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->page_size <= 0 || c->Hkv <= 0) return LCA_ERR_INVALID_ARG;
  if (c->d != kHeadDim || c->page_size % 8 != 0) return LCA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->n_pages) * c->page_size > 0x7FFFFFFFLL) return LCA_ERR_UNSUPPORTED;
  if (!stride_ok(c->page_stride) || !stride_ok(c->token_stride) || !stride_ok(c->head_stride))
    return LCA_ERR_INVALID_ARG;
  if (!fits(c->n_pages, c->page_stride) || !fits(c->page_size, c->token_stride) || !fits(c->Hkv, c->head_stride))
    return LCA_ERR_INVALID_ARG;
  return LCA_OK;
}

bool cache_memory(const lca_paged_cache* c) {
  if (c->n_pages == 0) return true;
  return c->k && c->v && aligned16(c->k) && aligned16(c->v) && device_input(c->k) && device_input(c->v);
}

// Bytes from the first to the last element of k, and of v.
long long cache_extent(const lca_paged_cache* c) {
  if (c->n_pages == 0) return 0;
  return ((c->n_pages - 1) * c->page_stride + (c->page_size - 1) * c->token_stride + (c->Hkv - 1) * c->head_stride +
          kHeadDim) * 2;
}

// The values' layout of an 8-bit cache, in elements.
lca_paged_cache values_of(const lca_paged_cache_fp8* c) {
  lca_paged_cache v{};
  if (c)
    v = {c->k, c->v, c->n_pages, c->page_size, c->Hkv, c->d, LCA_BF16, c->page_stride, c->token_stride, c->head_stride};
  return v;
}

lca_status check_cache8(const lca_paged_cache_fp8* c) {
  if (!c) return LCA_ERR_INVALID_ARG;
  const lca_paged_cache v = values_of(c);
  const lca_status r = check_cache(&v);
  if (r != LCA_OK) return r;
  if (c->Hkv > kMostHeads) return LCA_ERR_UNSUPPORTED;
  if (c->page_stride % 16 != 0 || c->token_stride % 16 != 0 || c->head_stride % 16 != 0) return LCA_ERR_INVALID_ARG;
  if (!stride_ok(c->scale_page_stride) || !stride_ok(c->scale_head_stride) || !fits(c->n_pages, c->scale_page_stride) ||
      !fits(c->Hkv, c->scale_head_stride))
    return LCA_ERR_INVALID_ARG;
  return LCA_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

bool cache_memory8(const lca_paged_cache_fp8* c) {
  if (c->n_pages == 0) return true;
  const lca_paged_cache v = values_of(c);
  return cache_memory(&v) && c->k_scale && c->v_scale && aligned8(c->k_scale) && aligned8(c->v_scale) &&
         device_input(c->k_scale) && device_input(c->v_scale);
}

// The four arrays of an 8-bit cache, from their first to their last byte.
struct Extent {
  const void* p;
  long long bytes;
};
void extents8(const lca_paged_cache_fp8* c, Extent (&e)[4]) {
  const lca_paged_cache v = values_of(c);
  const long long n = cache_extent(&v) / 2;
  const long long f = c->n_pages == 0 ? 0
                                      : (c->n_pages - 1) * c->scale_page_stride + (c->Hkv - 1) * c->scale_head_stride +
                                            c->page_size;
  e[0] = {c->k, n}, e[1] = {c->v, n}, e[2] = {c->k_scale, f}, e[3] = {c->v_scale, f};
}

// The cache's strides as a tensor map has them, in ascending order: token and
// head as they come, the page last.  The stride of an axis of length one moves
// nothing and is taken as its neighbour's.
struct MapStrides {
  int64_t token, head, page;
  bool head_first, ordered;
};
MapStrides map_strides(const lca_paged_cache* c) {
  MapStrides m;
  m.token = c->token_stride;
  m.head = c->Hkv > 1 ? c->head_stride : m.token;
  m.head_first = m.head < m.token;
  const int64_t most = m.head_first ? m.token : m.head;
  m.page = c->n_pages > 1 ? c->page_stride : most;
  m.ordered = m.page >= most;
  return m;
}

// Whether the kernel for many rows takes part: some request may have more
// rows per KV head than the other one's tile, a token's heads fit a tile, and
// there is a cache to map, its pages further apart than its tokens and heads.
// The other kernel reads a request's keys again for every 16 rows: 2048 tokens
// at 32K, 64 heads on 8, take 14.7 ms with heads or tokens as the outermost
// axis and 1.50 with pages; 512 at 8K with one group of 136 heads 2.06 ms, of
// 128 heads 0.22.
long long most_rows(const lca_paged_shape* sh, const lca_paged_cache* c) {  // of a request and KV head
  return static_cast<long long>(sh->max_q_len > 0 && sh->max_q_len < sh->Tq ? sh->max_q_len : sh->Tq) * (sh->Hq / c->Hkv);
}
bool many_rows(const lca_paged_shape* sh, const lca_paged_cache* c, bool eight) {
  return most_rows(sh, c) > (eight ? kPaged8FewRows : kPagedFewRows) && sh->Hq / c->Hkv <= kTile && c->n_pages > 0 &&
         map_strides(c).ordered;
}

int tokens_per_tile(const lca_paged_shape* sh, const lca_paged_cache* c) { return kTile / (sh->Hq / c->Hkv); }

struct PagedLayout {
  size_t status = 0, arrived = 0, parts = 0, block0 = 0, line = 0, cuts = 0, chunk_parts = 0, total = 0;
  int max_blocks = 0;
};

// Rows of an item of the kernel for few rows over an 8-bit cache (a 16-bit one's
// has 16): as many as the longest request has, or a single token where that one
// goes to the kernel for many rows (many).
int few_tile(const lca_paged_shape* sh, const lca_paged_cache* c, bool many) {
  const long long rows = many ? std::min<long long>(sh->Hq / c->Hkv, kPagedFewRows) : most_rows(sh, c);
  return static_cast<int>(rows >= kPaged8FewRows ? kPaged8FewRows : rows <= 8 ? 8 : (rows + 7) / 8 * 8);
}

PagedLayout paged_layout(const lca_paged_shape* sh, const lca_paged_cache* c, bool eight) {
  PagedLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  L.status = take(16);
  L.arrived = take(sizeof(int) * (kPagedMaxSpans + 1));
  const int rows = eight ? few_tile(sh, c, many_rows(sh, c, true)) : kPagedFewRows;
  L.parts = take(sizeof(float) * 2 * kPagedMaxSpans * rows * (kHeadDim + 2));
  if (many_rows(sh, c, eight)) {
    L.max_blocks = sh->Tq / (2 * tokens_per_tile(sh, c)) + sh->n_seq;
    L.block0 = take(sizeof(int) * (sh->n_seq + 1LL));
    L.line = take(sizeof(long long) * (L.max_blocks + 1LL));
    L.cuts = take(sizeof(PagedCut) * kPagedMaxChunkCtas);
    L.chunk_parts = take(sizeof(float) * 2 * kPagedMaxChunkCtas * kPagedChunkPartFloats);
  }
  L.total = o;
  return L;
}

// Whether a call over an 8-bit cache makes a 16-bit copy of its tables' pages
// first, on which its requests of many rows run (those of few stay with the 8-bit
// kernel and its items of 8 or 16 rows): it has so many rows per request that
// reading the keys as 8 bits costs more than the copy.  64 query heads on 8, as
// they are and copied: 2048 tokens at the end of 32K keys 1865 and 1565 us (33 of it
// the copy), 8 fresh prompts of 101-2047 tokens 460 and 307; 8 requests of 256, 192,
// 128 and 64 tokens at 16K keys 967 and 925, 737 and 727, 509 and 536, 275 and 352, at
// 1K keys 155 and 124, 122 and 103, 90 and 83, 59 and 62.
// Only for bf16 queries, whose copy holds every value as it is: fp16 ends at 65504
// and has nothing below 2^-24, and the same request must not get other scores for
// the rows that come with it (that chunk takes 1824 us, those prompts 448).
constexpr long long kCopyRows = 1536;
constexpr long long kCopyBytes = 1LL << 30;
long long copy_bytes(const lca_paged_shape* sh, const lca_paged_cache* c) {  // of K or V
  return static_cast<long long>(sh->n_seq) * sh->max_pages * c->page_size * c->Hkv * kHeadDim * 2;
}
bool copies(const lca_paged_shape* sh, const lca_paged_cache* c) {
  const long long n = sh->n_seq, hint = sh->max_q_len;
  const long long rows = hint > 0 && hint * n < sh->Tq ? hint * n : sh->Tq;
  // in doubles: none of these is small enough to multiply unseen
  const double bytes = static_cast<double>(n) * sh->max_pages * c->page_size * c->Hkv * kHeadDim * 4;
  return n > 0 && sh->max_pages > 0 && c->n_pages > 0 && bytes <= static_cast<double>(kCopyBytes) &&
         rows * (sh->Hq / c->Hkv) >= kCopyRows * n && static_cast<long long>(c->page_size) * c->Hkv <= 0x7FFFFF00LL &&
         sh->Hq / c->Hkv <= kTile;  // wider groups are not for the kernel that gains by it (many_rows)
}
// The copy's layout: [page of a table][head][token][128].
lca_paged_cache copy_of(const lca_paged_shape* sh, const lca_paged_cache* c, int dtype, uint8_t* at) {
  const int64_t head = static_cast<int64_t>(c->page_size) * kHeadDim;
  return {at, at + copy_bytes(sh, c), sh->n_seq * sh->max_pages, c->page_size, c->Hkv, kHeadDim, dtype, head * c->Hkv,
          kHeadDim, head};
}

// Workspace of a call over an 8-bit cache; where it copies, `copy` and `map` (the
// tables of the copy) lie behind what the call over the copy needs.
struct Layout8 {
  PagedLayout run;
  size_t copy = 0, map = 0, total = 0;
  bool copies = false;
};
Layout8 layout8(const lca_paged_shape* sh, const lca_paged_cache* c, bool bf16) {
  Layout8 L;
  L.copies = bf16 && copies(sh, c);
  if (!L.copies) {
    L.run = paged_layout(sh, c, true);
    L.total = L.run.total;
    return L;
  }
  const lca_paged_cache v = copy_of(sh, c, LCA_BF16, nullptr);
  L.run = paged_layout(sh, &v, false);
  L.copy = L.run.total;
  L.map = align_up(L.copy + 2 * static_cast<size_t>(copy_bytes(sh, c)));
  L.total = align_up(L.map + sizeof(int) * sh->n_seq * static_cast<size_t>(sh->max_pages));
  // a shorter longest request may make it a call without a copy
  const size_t other = paged_layout(sh, c, true).total;
  if (sh->max_q_len == 0 && other > L.total) L.total = other;
  return L;
}

lca_status check_attn(const lca_paged_shape* sh, const lca_paged_cache* c, const lca_mask_desc* md, MaskCtx& m) {
  if (!sh || !md) return LCA_ERR_INVALID_ARG;
  const lca_status r = check_cache(c);
  if (r != LCA_OK) return r;
  if (sh->Tq < 0 || sh->Hq <= 0 || sh->n_seq < 0 || sh->max_pages < 0 || sh->max_q_len < 0) return LCA_ERR_INVALID_ARG;
  if (sh->Hq % c->Hkv != 0) return LCA_ERR_INVALID_ARG;
  if (sh->n_seq > kMostRequests) return LCA_ERR_UNSUPPORTED;
  if (sh->table_stride < sh->max_pages || !fits(sh->n_seq, sh->table_stride)) return LCA_ERR_INVALID_ARG;
  if (sh->q_stride < static_cast<long long>(sh->Hq) * kHeadDim || !stride_ok(sh->q_stride) ||
      !fits(sh->Tq, sh->q_stride))
    return LCA_ERR_INVALID_ARG;
  if (!std::isfinite(sh->scale * 1.4426950408889634f) || sh->scale < 0.f) return LCA_ERR_INVALID_ARG;
  // sums of two lengths or of a length and a window stay in 32 bits, so do the launch grids
  if (static_cast<long long>(sh->max_pages) * c->page_size > 0x3FFFFF00LL || sh->Tq > 0x3FFFFFFF)
    return LCA_ERR_UNSUPPORTED;
  if (static_cast<long long>(sh->Tq) * sh->Hq > 0x7FFFFFFFLL || sh->Hq > kMostHeads) return LCA_ERR_UNSUPPORTED;
  m = MaskCtx{};
  m.kind = md->kind;
  m.wl = md->window_left;
  m.wr = md->window_right;
  m.ng = md->num_global;
  m.prefix = md->prefix_len;
  m.block = md->block;
  m.hm_count = 1;
  switch (md->kind) {
    case LCA_MASK_FULL:
    case LCA_MASK_DOC:
    case LCA_MASK_CAUSAL:
    case LCA_MASK_CAUSAL_DOC:
      break;
    case LCA_MASK_SLIDING:
    case LCA_MASK_CAUSAL_SLIDING:
    case LCA_MASK_GLOBAL_SLIDING:
      if (m.wl < 0 || m.wr < 0) return LCA_ERR_INVALID_ARG;
      if (md->kind == LCA_MASK_GLOBAL_SLIDING && m.ng < 0) return LCA_ERR_INVALID_ARG;
      break;
    case LCA_MASK_PREFIX_LM_CAUSAL:
      if (m.prefix < 0) return LCA_ERR_INVALID_ARG;
      break;
    case LCA_MASK_CAUSAL_BLOCKWISE:
    case LCA_MASK_BLOCK_CAUSAL_DOC:
      if (m.block < 1) return LCA_ERR_INVALID_ARG;
      break;
    case LCA_MASK_SHARED_QUESTION:
    case LCA_MASK_PREFIX_LM_DOC:
    case LCA_MASK_BLOCK_SPARSE_UNIFORM:
    case LCA_MASK_BLOCK_SPARSE_VARIABLE:
    case LCA_MASK_FLASHMASK:
      return LCA_ERR_UNSUPPORTED;
    default:
      return LCA_ERR_INVALID_ARG;
  }
  // a distance or block beyond every length acts as that length; keeping it
  // there keeps position arithmetic in 32 bits
  constexpr int kFar = 0x3FFFFFFF;
  m.wl = m.wl < kFar ? m.wl : kFar;
  m.wr = m.wr < kFar ? m.wr : kFar;
  m.block = m.block < kFar ? m.block : kFar;
  return LCA_OK;
}

bool encode(CUtensorMap* m, const void* p, CUtensorMapDataType type, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const auto fn = encode_fn();
  if (!fn) {
    driver_fail("cuTensorMapEncodeTiled entry point", 0);
    return false;
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, type, rank, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) driver_fail("cuTensorMapEncodeTiled", static_cast<int>(r));
  return r == CUDA_SUCCESS;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == LCA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Boxes of box_rows rows of 128 bytes.
bool cache_map(CUtensorMap* m, const void* p, const Cache& any, int box_rows) {
  const lca_paged_cache* c = any.c;
  const cuuint64_t bytes = static_cast<cuuint64_t>(any.bytes());
  const MapStrides st = map_strides(c);
  const bool hf = st.head_first;
  const cuuint64_t tokens = static_cast<cuuint64_t>(c->page_size), heads = static_cast<cuuint64_t>(c->Hkv);
  const cuuint64_t dims[4] = {kHeadDim, hf ? heads : tokens, hf ? tokens : heads, static_cast<cuuint64_t>(c->n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(hf ? st.head : st.token) * bytes,
                                 static_cast<cuuint64_t>(hf ? st.token : st.head) * bytes,
                                 static_cast<cuuint64_t>(st.page) * bytes};
  const cuuint32_t rows = static_cast<cuuint32_t>(box_rows);
  const cuuint32_t box[4] = {any.c8 ? 128u : 64u, hf ? 1 : rows, hf ? rows : 1, 1};
  return encode(m, p, any.c8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : map_type(c->dtype), 4, dims, strides, box);
}

// What the kernel that reads pages back needs to know of a cache and its copy.
void read_args(const lca_paged_cache_fp8* cache, const lca_paged_cache* out, PagedRead8Args& a) {
  a.kc = static_cast<const uint8_t*>(cache->k);
  a.vc = static_cast<const uint8_t*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.k = static_cast<uint16_t*>(out->k);
  a.v = static_cast<uint16_t*>(out->v);
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.scale_page_stride = cache->scale_page_stride;
  a.scale_head_stride = cache->scale_head_stride;
  a.out_page_stride = out->page_stride;
  a.out_token_stride = out->token_stride;
  a.out_head_stride = out->head_stride;
  a.n_pages = cache->n_pages;
  a.Hkv = cache->Hkv;
  a.page_size = cache->page_size;
  a.token_first = cache->token_stride < cache->head_stride;
  a.out_v8 = ((reinterpret_cast<uintptr_t>(out->k) | reinterpret_cast<uintptr_t>(out->v)) & 31u) == 0 &&
             out->page_stride % 16 == 0 && out->token_stride % 16 == 0 && out->head_stride % 16 == 0;
}

// What divides a key's index by the page size as a product: with 2^s the power of
// two at or above page_size and mul = ceil(2^(30 + s) / page_size), which is
// less than 2^31 + 1, mul page_size passes 2^(30 + s) by less than 2^s, so
// floor(j mul / 2^(30 + s)) is exact for j < 2^30.
void page_divisor(PagedAttnArgs& a) {
  int s = 3;
  while ((1LL << s) < a.page_size) ++s;
  a.page_mul = static_cast<uint32_t>(((1ULL << (30 + s)) + a.page_size - 1) / a.page_size);
  a.page_shift = s - 2;
}

// lca_attn_paged over a cache of either kind, q and o of `dtype`.
lca_status attend(const Cache& any, int dtype, const void* q, const int32_t* block_table, const int32_t* q_start,
                  const int32_t* k_len, void* o, float* lse, const lca_paged_shape* shape, const lca_mask_desc* mask,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const lca_paged_cache* cache = any.c;
  const lca_paged_cache_fp8* c8 = any.c8;
  PagedAttnArgs a{};
  const lca_status r = check_attn(shape, cache, mask, a.mask);
  if (r != LCA_OK) return r;
  Layout8 L8;
  if (c8) {
    L8 = layout8(shape, cache, dtype == LCA_BF16);
  } else {
    L8.run = paged_layout(shape, cache, false);
    L8.total = L8.run.total;
  }
  const PagedLayout& L = L8.run;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 || workspace_bytes < L8.total ||
      !device_input(workspace))
    return LCA_ERR_WORKSPACE;
  const long long n_table =
      shape->n_seq > 0 && shape->max_pages > 0 ? (shape->n_seq - 1) * shape->table_stride + shape->max_pages : 0;
  if (!ints(block_table, n_table) || !ints(q_start, shape->n_seq > 0 ? shape->n_seq + 1LL : 0) ||
      !ints(k_len, shape->n_seq) || (shape->ctx_len && !ints(shape->ctx_len, shape->n_seq)) || !(c8 ? cache_memory8(c8) : cache_memory(cache)))
    return LCA_ERR_INVALID_ARG;
  if (shape->Tq > 0) {
    if (!q || !aligned16(q) || !device_input(q) || !o || !aligned16(o) || !device_input(o) || !lse || !aligned4(lse) ||
        !device_input(lse))
      return LCA_ERR_INVALID_ARG;
  }
  {  // an empty batch writes its workspace too
    const long long rows = shape->Tq, heads = shape->Hq;
    const long long extent = cache_extent(cache) / 2 * any.bytes();
    Extent e8[4] = {};
    if (c8) extents8(c8, e8);
    const Extent t[12] = {{o, rows * heads * kHeadDim * 2},
              {lse, rows * heads * 4},
              {workspace, static_cast<long long>(L8.total)},
              {q, rows > 0 ? ((rows - 1) * shape->q_stride + heads * kHeadDim) * 2 : 0},
              {cache->k, extent},
              {cache->v, extent},
              {block_table, 4 * n_table},
              {q_start, 4 * (shape->n_seq + 1LL)},
              {k_len, 4LL * shape->n_seq},
              {shape->ctx_len, shape->ctx_len ? 4LL * shape->n_seq : 0},
              e8[2],
              e8[3]};
    for (int i = 0; i < 3; ++i)  // the first three are written
      for (int j = i + 1; j < 12; ++j)
        if (overlap(t[i].p, t[i].bytes, t[j].p, t[j].bytes)) return LCA_ERR_INVALID_ARG;
  }
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fp16 = dtype == LCA_F16;
  a.table_stride = shape->table_stride;
  a.table = block_table;
  a.q_start = q_start;
  a.k_len = k_len;
  a.ctx_len = shape->ctx_len;
  a.Tq = shape->Tq;
  a.n_seq = shape->n_seq;
  a.max_pages = shape->max_pages;
  a.page_size = cache->page_size;
  page_divisor(a);
  a.q = q;
  a.q_stride = shape->q_stride;
  a.o = o;
  a.lse = lse;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.arrived = reinterpret_cast<int*>(ws + L.arrived);
  a.claims = a.arrived + kPagedMaxSpans;
  a.parts = reinterpret_cast<float*>(ws + L.parts);
  a.Hq = shape->Hq;
  a.Hkv = cache->Hkv;
  a.G = shape->Hq / cache->Hkv;
  const float scale = shape->scale > 0.f ? shape->scale : 1.0f / std::sqrt(static_cast<float>(kHeadDim));
  a.scale_log2 = scale * 1.4426950408889634f;
  auto over = [&](const Cache& x) {
    a.kc = x.c->k;
    a.vc = x.c->v;
    a.page_stride = x.c->page_stride;
    a.token_stride = x.c->token_stride;
    a.head_stride = x.c->head_stride;
    a.n_pages = x.c->n_pages;
    if (x.c8) {
      a.ks = x.c8->k_scale;
      a.vs = x.c8->v_scale;
      a.scale_page_stride = x.c8->scale_page_stride;
      a.scale_head_stride = x.c8->scale_head_stride;
    }
    if (x.c->n_pages == 0) {  // no key is read; the addresses are only given
      a.kc = a.vc = q;
      a.ks = a.vs = static_cast<const uint8_t*>(q);
    }
  };
  over(any);
  // with a copy the kernel for many rows has other arguments than the one for few
  Cache run = any;
  lca_paged_cache copy{};
  if (L8.copies) {
    copy = copy_of(shape, cache, dtype, ws + L8.copy);
    run = {&copy, nullptr};
  }
  const bool many = many_rows(shape, run.c, run.c8 != nullptr) && shape->n_seq > 0;
  a.few = many ? kPagedFewRows : 0x7FFFFFFF;
  const PagedAttnArgs direct = a;
  if (L8.copies) {
    PagedRead8Args c{};
    read_args(c8, &copy, c);
    c.n = copy.n_pages;
    int* map = reinterpret_cast<int*>(ws + L8.map);
    launch_paged_copy8(c, a, map, fp16, sms, st);
    LCA_CUDA(cudaGetLastError());
    over(run);
    a.table = map;
    a.table_stride = shape->max_pages;
  }
  CUtensorMap tq, tk, tv;
  if (many) {
    a.tpt = tokens_per_tile(shape, cache);
    a.box_rows = kTile;
    while (cache->page_size % a.box_rows != 0) a.box_rows /= 2;
    a.head_first = map_strides(run.c).head_first;
    a.max_blocks = L.max_blocks;
    a.block0 = reinterpret_cast<int*>(ws + L.block0);
    a.line = reinterpret_cast<long long*>(ws + L.line);
    a.cuts = reinterpret_cast<PagedCut*>(ws + L.cuts);
    a.chunk_parts = reinterpret_cast<float*>(ws + L.chunk_parts);
    a.out_v8 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
    a.wait_limit_ns = wait_limit_ns();
    const cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.Tq)};
    const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(a.tpt)};
    if (!encode(&tq, q, map_type(dtype), 3, dims, strides, box) || !cache_map(&tk, run.c->k, run, a.box_rows) ||
        !cache_map(&tv, run.c->v, run, a.box_rows))
      return LCA_ERR_CUDA;
  }
  LCA_CUDA(launch_paged_begin(a, many, st));
  if (many) LCA_CUDA((run.c8 ? launch_paged_chunk8 : launch_paged_chunk)(tq, tk, tv, a, fp16, sms, st));
  if (shape->Tq > 0)
    LCA_CUDA(c8 ? launch_paged_decode8(direct, few_tile(shape, cache, many), many, fp16, sms, st)
                : launch_paged_decode(direct, many, fp16, sms, st));
  if (many) LCA_CUDA(launch_paged_join(a, fp16, run.c8 != nullptr, sms, st));
  return LCA_OK;
}

}  // namespace
}  // namespace lca

using namespace lca;

extern "C" {

lca_status lca_paged_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t n_seq, const int32_t* free_pages,
                          int32_t n_free, const int32_t* taken, int32_t* block_table, int64_t table_stride,
                          int32_t max_pages, int32_t page_size, int32_t n_pages, int32_t n_rows, int32_t* q_start,
                          int32_t* k_len, int32_t* slots, int32_t* positions, int32_t* state, void* stream) {
  if (n_seq < 0 || n_free < 0 || max_pages < 0 || page_size <= 0 || n_pages < 0 || n_rows < 0 ||
      table_stride < max_pages || !fits(n_seq, table_stride))
    return LCA_ERR_INVALID_ARG;
  if (static_cast<long long>(n_pages) * page_size > 0x7FFFFFFFLL ||
      static_cast<long long>(max_pages) * page_size > 0x7FFFFF00LL || n_seq > kMostRequests)
    return LCA_ERR_UNSUPPORTED;
  const long long n_table = n_seq > 0 && max_pages > 0 ? (n_seq - 1) * table_stride + max_pages : 0;
  if (!ints(ctx_len, n_seq) || !ints(new_len, n_seq) || !ints(free_pages, n_free) || !ints(taken, 1) ||
      !ints(block_table, n_table) || !ints(q_start, n_seq + 1LL) || !ints(k_len, n_seq) || !ints(slots, n_rows) ||
      !ints(positions, n_rows) || !ints(state, 4))
    return LCA_ERR_INVALID_ARG;
  const struct {
    const void* p;
    long long bytes;
  } t[10] = {{q_start, 4 * (n_seq + 1LL)}, {k_len, 4LL * n_seq}, {slots, 4LL * n_rows},   {positions, 4LL * n_rows},
             {state, 16},                  {block_table, 4 * n_table}, {ctx_len, 4LL * n_seq}, {new_len, 4LL * n_seq},
             {free_pages, 4LL * n_free},   {taken, 4}};
  for (int i = 0; i < 6; ++i)  // the first six are written
    for (int j = i + 1; j < 10; ++j)
      if (overlap(t[i].p, t[i].bytes, t[j].p, t[j].bytes)) return LCA_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  const PagedPlanArgs a{ctx_len, new_len, free_pages, taken,   block_table, table_stride, n_seq, n_free,    max_pages,
                        page_size, n_pages, n_rows,   q_start, k_len,       slots,        positions, state};
  launch_paged_plan(a, sms, static_cast<cudaStream_t>(stream));
  LCA_CUDA(cudaGetLastError());
  return LCA_OK;
}

lca_status lca_paged_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
                           int32_t n_rows, const lca_paged_cache* cache, void* stream) {
  const lca_status r = check_cache(cache);
  if (r != LCA_OK) return r;
  const long long row = static_cast<long long>(cache->Hkv) * kHeadDim;
  if (n_rows < 0 || k_stride < row || v_stride < row || !stride_ok(k_stride) || !stride_ok(v_stride) ||
      !fits(n_rows, k_stride) || !fits(n_rows, v_stride))
    return LCA_ERR_INVALID_ARG;
  if (n_rows == 0) return LCA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !device_input(k) || !device_input(v) || !ints(slots, n_rows))
    return LCA_ERR_INVALID_ARG;
  if (cache->n_pages == 0) return LCA_OK;  // every slot lies outside
  if (!cache_memory(cache)) return LCA_ERR_INVALID_ARG;
  for (const void* c : {cache->k, cache->v}) {
    const long long n = cache_extent(cache);
    if (overlap(c, n, k, ((n_rows - 1) * k_stride + row) * 2) || overlap(c, n, v, ((n_rows - 1) * v_stride + row) * 2) ||
        overlap(c, n, slots, 4LL * n_rows))
      return LCA_ERR_INVALID_ARG;
  }
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  PagedWriteArgs a{};
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.kc = static_cast<uint4*>(cache->k);
  a.vc = static_cast<uint4*>(cache->v);
  a.k_stride = k_stride / 8;
  a.v_stride = v_stride / 8;
  a.page_stride = cache->page_stride / 8;
  a.token_stride = cache->token_stride / 8;
  a.head_stride = cache->head_stride / 8;
  a.slots = slots;
  a.n_rows = n_rows;
  a.Hkv = cache->Hkv;
  a.page_size = cache->page_size;
  a.n_slots = cache->n_pages * cache->page_size;
  launch_paged_write(a, sms, static_cast<cudaStream_t>(stream));
  LCA_CUDA(cudaGetLastError());
  return LCA_OK;
}

lca_status lca_paged_write_fp8(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int32_t dtype,
                               const int32_t* slots, int32_t n_rows, const lca_paged_cache_fp8* cache, void* stream) {
  const lca_status r = check_cache8(cache);
  if (r != LCA_OK) return r;
  if (dtype != LCA_BF16 && dtype != LCA_F16) return LCA_ERR_INVALID_ARG;
  const long long row = static_cast<long long>(cache->Hkv) * kHeadDim;
  if (n_rows < 0 || k_stride < row || v_stride < row || !stride_ok(k_stride) || !stride_ok(v_stride) ||
      !fits(n_rows, k_stride) || !fits(n_rows, v_stride))
    return LCA_ERR_INVALID_ARG;
  if (n_rows == 0) return LCA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !device_input(k) || !device_input(v) || !ints(slots, n_rows))
    return LCA_ERR_INVALID_ARG;
  if (cache->n_pages == 0) return LCA_OK;  // every slot lies outside
  if (!cache_memory8(cache)) return LCA_ERR_INVALID_ARG;
  Extent e[4];
  extents8(cache, e);
  for (const Extent& c : e)
    if (overlap(c.p, c.bytes, k, ((n_rows - 1) * k_stride + row) * 2) ||
        overlap(c.p, c.bytes, v, ((n_rows - 1) * v_stride + row) * 2) || overlap(c.p, c.bytes, slots, 4LL * n_rows))
      return LCA_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  PagedWrite8Args a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.kc = static_cast<uint8_t*>(cache->k);
  a.vc = static_cast<uint8_t*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.scale_page_stride = cache->scale_page_stride;
  a.scale_head_stride = cache->scale_head_stride;
  a.slots = slots;
  a.n_rows = n_rows;
  a.Hkv = cache->Hkv;
  a.page_size = cache->page_size;
  a.n_slots = cache->n_pages * cache->page_size;
  a.in_v8 = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0 && k_stride % 16 == 0 &&
            v_stride % 16 == 0;
  launch_paged_write8(a, dtype == LCA_F16, sms, static_cast<cudaStream_t>(stream));
  LCA_CUDA(cudaGetLastError());
  return LCA_OK;
}

lca_status lca_paged_read_fp8(const lca_paged_cache_fp8* cache, const int32_t* pages, int32_t n,
                              const lca_paged_cache* out, void* stream) {
  lca_status r = check_cache8(cache);
  if (r == LCA_OK) r = check_cache(out);
  if (r != LCA_OK) return r;
  if (n < 0 || n > out->n_pages || out->page_size != cache->page_size || out->Hkv != cache->Hkv)
    return LCA_ERR_INVALID_ARG;
  if (n == 0) return LCA_OK;
  if (static_cast<long long>(cache->page_size) * cache->Hkv > 0x7FFFFF00LL) return LCA_ERR_UNSUPPORTED;
  if (!ints(pages, n) || !cache_memory(out)) return LCA_ERR_INVALID_ARG;
  if (cache->n_pages == 0) return LCA_OK;  // every entry lies outside
  if (!cache_memory8(cache)) return LCA_ERR_INVALID_ARG;
  Extent e[4];
  extents8(cache, e);
  for (const void* p : {out->k, out->v}) {
    const long long bytes = cache_extent(out);
    if (overlap(p, bytes, pages, 4LL * n)) return LCA_ERR_INVALID_ARG;
    for (const Extent& c : e)
      if (overlap(p, bytes, c.p, c.bytes)) return LCA_ERR_INVALID_ARG;
  }
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  PagedRead8Args a{};
  read_args(cache, out, a);
  a.pages = pages;
  a.n = n;
  launch_paged_read8(a, out->dtype == LCA_F16, sms, static_cast<cudaStream_t>(stream));
  LCA_CUDA(cudaGetLastError());
  return LCA_OK;
}

lca_status lca_attn_paged_workspace_size(const lca_paged_shape* shape, const lca_paged_cache* cache,
                                         const lca_mask_desc* mask, size_t* bytes) {
  if (!bytes) return LCA_ERR_INVALID_ARG;
  MaskCtx m;
  const lca_status r = check_attn(shape, cache, mask, m);
  if (r != LCA_OK) return r;
  *bytes = paged_layout(shape, cache, false).total;
  return LCA_OK;
}

lca_status lca_attn_paged(const void* q, const lca_paged_cache* cache, const int32_t* block_table,
                          const int32_t* q_start, const int32_t* k_len, void* o, float* lse,
                          const lca_paged_shape* shape, const lca_mask_desc* mask, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return attend({cache, nullptr}, cache ? cache->dtype : 0, q, block_table, q_start, k_len, o, lse, shape, mask, workspace,
                workspace_bytes, stream);
}

lca_status lca_attn_paged_fp8_workspace_size(const lca_paged_shape* shape, const lca_paged_cache_fp8* cache,
                                             const lca_mask_desc* mask, size_t* bytes) {
  lca_status r = check_cache8(cache);
  if (r != LCA_OK) return r;
  if (!bytes) return LCA_ERR_INVALID_ARG;
  const lca_paged_cache v = values_of(cache);
  MaskCtx m;
  r = check_attn(shape, &v, mask, m);
  if (r != LCA_OK) return r;
  *bytes = std::max(layout8(shape, &v, true).total, layout8(shape, &v, false).total);  // q's type is not known here
  return LCA_OK;
}

lca_status lca_attn_paged_fp8(const void* q, int32_t dtype, const lca_paged_cache_fp8* cache, const int32_t* block_table,
                              const int32_t* q_start, const int32_t* k_len, void* o, float* lse,
                              const lca_paged_shape* shape, const lca_mask_desc* mask, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const lca_status r = check_cache8(cache);
  if (r != LCA_OK) return r;
  if (dtype != LCA_BF16 && dtype != LCA_F16) return LCA_ERR_INVALID_ARG;
  const lca_paged_cache v = values_of(cache);
  return attend({&v, cache}, dtype, q, block_table, q_start, k_len, o, lse, shape, mask, workspace, workspace_bytes,
                stream);
}

}  // extern "C"
