// lca_paged_api.cu — the paged-cache entry points of include/lca_attn.h:
// argument checks (all before anything is launched), workspace layout and
// launches.  Nothing here allocates or throws.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>

#include "../../include/lca_attn.h"
#include "lca_host.h"
#include "lca_paged.h"

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
bool many_rows(const lca_paged_shape* sh, const lca_paged_cache* c) {
  const long long G = sh->Hq / c->Hkv;
  const long long most = sh->max_q_len > 0 && sh->max_q_len < sh->Tq ? sh->max_q_len : sh->Tq;
  return most * G > kPagedFewRows && G <= kTile && c->n_pages > 0 && map_strides(c).ordered;
}

int tokens_per_tile(const lca_paged_shape* sh, const lca_paged_cache* c) { return kTile / (sh->Hq / c->Hkv); }

struct PagedLayout {
  size_t status = 0, arrived = 0, parts = 0, block0 = 0, line = 0, cuts = 0, chunk_parts = 0, total = 0;
  int max_blocks = 0;
};

PagedLayout paged_layout(const lca_paged_shape* sh, const lca_paged_cache* c) {
  PagedLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  L.status = take(16);
  L.arrived = take(sizeof(int) * (kPagedMaxSpans + 1));
  L.parts = take(sizeof(float) * 2 * kPagedMaxSpans * kPagedPartFloats);
  if (many_rows(sh, c)) {
    L.max_blocks = sh->Tq / (2 * tokens_per_tile(sh, c)) + sh->n_seq;
    L.block0 = take(sizeof(int) * (sh->n_seq + 1LL));
    L.line = take(sizeof(long long) * (L.max_blocks + 1LL));
    L.cuts = take(sizeof(PagedCut) * kPagedMaxChunkCtas);
    L.chunk_parts = take(sizeof(float) * 2 * kPagedMaxChunkCtas * kPagedChunkPartFloats);
  }
  L.total = o;
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
  if (static_cast<long long>(sh->Tq) * sh->Hq > 0x7FFFFFFFLL) return LCA_ERR_UNSUPPORTED;
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

bool encode(CUtensorMap* m, const void* p, int dtype, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const auto fn = encode_fn();
  if (!fn) {
    driver_fail("cuTensorMapEncodeTiled entry point", 0);
    return false;
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, dtype == LCA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                        const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) driver_fail("cuTensorMapEncodeTiled", static_cast<int>(r));
  return r == CUDA_SUCCESS;
}

bool cache_map(CUtensorMap* m, const void* p, const lca_paged_cache* c, int box_rows) {
  const MapStrides st = map_strides(c);
  const bool hf = st.head_first;
  const cuuint64_t tokens = static_cast<cuuint64_t>(c->page_size), heads = static_cast<cuuint64_t>(c->Hkv);
  const cuuint64_t dims[4] = {kHeadDim, hf ? heads : tokens, hf ? tokens : heads, static_cast<cuuint64_t>(c->n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(hf ? st.head : st.token) * 2,
                                 static_cast<cuuint64_t>(hf ? st.token : st.head) * 2,
                                 static_cast<cuuint64_t>(st.page) * 2};
  const cuuint32_t rows = static_cast<cuuint32_t>(box_rows);
  const cuuint32_t box[4] = {64, hf ? 1 : rows, hf ? rows : 1, 1};
  return encode(m, p, c->dtype, 4, dims, strides, box);
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

lca_status lca_attn_paged_workspace_size(const lca_paged_shape* shape, const lca_paged_cache* cache,
                                         const lca_mask_desc* mask, size_t* bytes) {
  if (!bytes) return LCA_ERR_INVALID_ARG;
  MaskCtx m;
  const lca_status r = check_attn(shape, cache, mask, m);
  if (r != LCA_OK) return r;
  *bytes = paged_layout(shape, cache).total;
  return LCA_OK;
}

lca_status lca_attn_paged(const void* q, const lca_paged_cache* cache, const int32_t* block_table,
                          const int32_t* q_start, const int32_t* k_len, void* o, float* lse,
                          const lca_paged_shape* shape, const lca_mask_desc* mask, void* workspace,
                          size_t workspace_bytes, void* stream) {
  PagedAttnArgs a{};
  const lca_status r = check_attn(shape, cache, mask, a.mask);
  if (r != LCA_OK) return r;
  const PagedLayout L = paged_layout(shape, cache);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 || workspace_bytes < L.total ||
      !device_input(workspace))
    return LCA_ERR_WORKSPACE;
  const long long n_table =
      shape->n_seq > 0 && shape->max_pages > 0 ? (shape->n_seq - 1) * shape->table_stride + shape->max_pages : 0;
  if (!ints(block_table, n_table) || !ints(q_start, shape->n_seq > 0 ? shape->n_seq + 1LL : 0) ||
      !ints(k_len, shape->n_seq) || (shape->ctx_len && !ints(shape->ctx_len, shape->n_seq)) || !cache_memory(cache))
    return LCA_ERR_INVALID_ARG;
  if (shape->Tq > 0) {
    if (!q || !aligned16(q) || !device_input(q) || !o || !aligned16(o) || !device_input(o) || !lse || !aligned4(lse) ||
        !device_input(lse))
      return LCA_ERR_INVALID_ARG;
  }
  {  // an empty batch writes its workspace too
    const long long rows = shape->Tq, heads = shape->Hq;
    const long long extent = cache_extent(cache);
    const struct {
      const void* p;
      long long bytes;
    } t[10] = {{o, rows * heads * kHeadDim * 2},
              {lse, rows * heads * 4},
              {workspace, static_cast<long long>(L.total)},
              {q, rows > 0 ? ((rows - 1) * shape->q_stride + heads * kHeadDim) * 2 : 0},
              {cache->k, extent},
              {cache->v, extent},
              {block_table, 4 * n_table},
              {q_start, 4 * (shape->n_seq + 1LL)},
              {k_len, 4LL * shape->n_seq},
              {shape->ctx_len, shape->ctx_len ? 4LL * shape->n_seq : 0}};
    for (int i = 0; i < 3; ++i)  // the first three are written
      for (int j = i + 1; j < 10; ++j)
        if (overlap(t[i].p, t[i].bytes, t[j].p, t[j].bytes)) return LCA_ERR_INVALID_ARG;
  }
  const int sms = num_sms();
  if (sms <= 0) return LCA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = q;
  a.kc = cache->k;
  a.vc = cache->v;
  a.q_stride = shape->q_stride;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.table_stride = shape->table_stride;
  a.table = block_table;
  a.q_start = q_start;
  a.k_len = k_len;
  a.ctx_len = shape->ctx_len;
  a.o = o;
  a.lse = lse;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.arrived = reinterpret_cast<int*>(ws + L.arrived);
  a.claims = a.arrived + kPagedMaxSpans;
  a.parts = reinterpret_cast<float*>(ws + L.parts);
  a.Tq = shape->Tq;
  a.Hq = shape->Hq;
  a.Hkv = cache->Hkv;
  a.G = shape->Hq / cache->Hkv;
  a.n_seq = shape->n_seq;
  a.max_pages = shape->max_pages;
  a.page_size = cache->page_size;
  a.n_pages = cache->n_pages;
  const float scale = shape->scale > 0.f ? shape->scale : 1.0f / std::sqrt(static_cast<float>(kHeadDim));
  a.scale_log2 = scale * 1.4426950408889634f;
  if (cache->n_pages == 0) a.kc = a.vc = q;  // no key is read; the address is only given
  const bool many = many_rows(shape, cache) && shape->n_seq > 0;
  a.few = many ? kPagedFewRows : 0x7FFFFFFF;
  CUtensorMap tq, tk, tv;
  if (many) {
    a.tpt = tokens_per_tile(shape, cache);
    a.box_rows = kTile;
    while (cache->page_size % a.box_rows != 0) a.box_rows /= 2;
    a.head_first = map_strides(cache).head_first;
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
    if (!encode(&tq, q, cache->dtype, 3, dims, strides, box) || !cache_map(&tk, cache->k, cache, a.box_rows) ||
        !cache_map(&tv, cache->v, cache, a.box_rows))
      return LCA_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fp16 = cache->dtype == LCA_F16;
  LCA_CUDA(launch_paged_begin(a, many, st));
  if (many) LCA_CUDA(launch_paged_chunk(tq, tk, tv, a, fp16, sms, st));
  if (shape->Tq > 0) LCA_CUDA(launch_paged_decode(a, many, fp16, sms, st));
  if (many) LCA_CUDA(launch_paged_join(a, fp16, sms, st));
  return LCA_OK;
}

}  // extern "C"
