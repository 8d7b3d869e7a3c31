/* lca_attn.h — C ABI of the GB300 (sm_103a) masked core-attention library.
 *
 * What it computes.  Core attention softmax(Q K^T * scale) V, forward and
 * backward, as defined on the FlashAttention review page
 * ("长上下文能力：FlashAttention vs. RingAttention", FlashAttention-1
 * 问题和瓶颈), computed IO-aware (FlashAttention-1 核心优化: tiling, online
 * softmax, fusion; FlashAttention-2 核心优化: deferred rescaling, one stored
 * row statistic, sequence-parallel work split), under the mask families of
 * the LongCA-bench review ("Long-Context Attention Benchmark", 三 技术架构,
 * 掩码模式分类), over packed batches of token-level shards of arbitrary
 * length ("Efficient Long-context Language Model Training by Core Attention
 * Disaggregation", 方法详解: stateless, composable core attention).
 *
 * Conventions shared by every entry point.
 *  - Tensors are token-major packed, row-major, bf16 unless stated:
 *      Q, O, dO, dQ : [Tq][Hq][d]        K, V, dK, dV : [Tk][Hkv][d]
 *      LSE          : [Hq][Tq] float32, natural log; -inf for a row with no key
 *    d must be 128.  Query head h reads KV head h / (Hq / Hkv).
 *  - Work is described by segments: query rows [q_off, q_off+q_len) attend
 *    keys [k_off, k_off+k_len).  A plain batch is B equal segments, a
 *    document-packed sequence one segment per document, a shard batch one
 *    segment per shard with k_off = its document's start and k_len = the
 *    shard's end within the document.  Causal families align the diagonal
 *    bottom-right (query i sits at key position i + k_len - q_len).
 *    Segments' query ranges must not overlap.  Segments with the same k_off
 *    form a key group; different key groups' key ranges must not overlap.
 *    Query rows outside every segment get O = 0, LSE = -inf, dQ = 0; keys
 *    outside every segment get dK = dV = 0.
 *  - The caller owns every buffer.  Pointers documented "device" are CUDA
 *    device pointers; "host" pointers are read during the call only.  The
 *    calls allocate no device memory: they take a caller-provided workspace
 *    of at least lca_workspace_size() bytes, 256-byte aligned.  (The one
 *    static array of lca_attn_fwd_static_workspace is reserved by CUDA when
 *    it loads this library's device code on a device; see there.)
 *  - Every device pointer must belong to the device that is current when the
 *    call is made (or be managed memory); the stream must belong to that
 *    device too.  A pointer to another device's memory is refused with
 *    LCA_ERR_INVALID_ARG before anything is launched.
 *  - The outputs of lca_attn_fwd (o, lse) and lca_attn_bwd (dq, dk, dv) may
 *    also be page-locked host memory that CUDA maps for the device
 *    (cudaMallocHost, cudaHostAlloc, or cudaHostRegister with mapping): the
 *    kernels store the results into it directly, which on a GB300 goes over
 *    NVLink-C2C to the Grace host's memory and needs no copy afterwards.
 *    Inputs and the workspace must be device (or managed) memory.  The
 *    library asks CUDA what each pointer is before launching: a pointer of
 *    another kind (pageable host memory, an unknown address) makes the call
 *    return LCA_ERR_INVALID_ARG (LCA_ERR_WORKSPACE for the workspace).
 *  - Calls are asynchronous on `stream` and never synchronise, except
 *    lca_read_status.  Argument errors are returned before anything is
 *    launched.  Faults detected on the device (a bounded wait that ran out,
 *    a block index out of range) are recorded in a status word inside the
 *    workspace and read with lca_read_status.
 */
#ifndef LCA_ATTN_H
#define LCA_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LCA_API __attribute__((visibility("default")))
#else
#define LCA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LCA_OK = 0,
  LCA_ERR_INVALID_ARG = 1, /* malformed shape, segments or mask descriptor   */
  LCA_ERR_UNSUPPORTED = 2, /* well-formed but outside what the kernels cover */
  LCA_ERR_WORKSPACE = 3,   /* workspace null, misaligned or too small        */
  LCA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed              */
  LCA_ERR_TIMEOUT = 5,     /* device: a bounded pipeline wait ran out        */
  LCA_ERR_DEVICE_ARG = 6   /* device: descriptor data out of range           */
} lca_status;

/* Mask families (LongCA-bench review, 三 技术架构, 掩码模式分类).  i and j are
 * positions inside a segment, ie = i + k_len - q_len.  Readings of the
 * unnamed details are stated per family. */
typedef enum {
  LCA_MASK_FULL = 0,             /* every key                                          */
  LCA_MASK_CAUSAL = 1,           /* j <= ie                                            */
  LCA_MASK_SLIDING = 2,          /* ie - window_left <= j <= ie + window_right          */
  LCA_MASK_CAUSAL_SLIDING = 3,   /* ie - window_left <= j <= ie                         */
  LCA_MASK_DOC = 4,              /* FULL inside each segment (segment = document)      */
  LCA_MASK_CAUSAL_DOC = 5,       /* CAUSAL inside each segment                         */
  LCA_MASK_SHARED_QUESTION = 6,  /* j <= ie and (part(j) == 0 or part(j) == part(ie));
                                    part 0 = question, parts from part_bounds          */
  LCA_MASK_GLOBAL_SLIDING = 7,   /* ie < num_global or j < num_global or
                                    ie - window_left <= j <= ie + window_right          */
  LCA_MASK_CAUSAL_BLOCKWISE = 8, /* j <= ie and (j/block == ie/block or
                                    ie/block == (k_len-1)/block)                       */
  LCA_MASK_PREFIX_LM_CAUSAL = 9, /* j < prefix_len or j <= ie                          */
  LCA_MASK_PREFIX_LM_DOC = 10,   /* j < seg_prefix[segment] or j <= ie                 */
  LCA_MASK_BLOCK_CAUSAL_DOC = 11,/* floor(j/block) <= floor(ie/block)                  */
  LCA_MASK_BLOCK_SPARSE_UNIFORM = 12,  /* keep[h][qb][kb], blocks q_block x kv_block  */
  LCA_MASK_BLOCK_SPARSE_VARIABLE = 13, /* keep[h][qb][kb], blocks from qb/kb_bounds   */
  LCA_MASK_FLASHMASK = 14  /* column-wise (FlashMask, named by the LongCA-bench review as
                              covering every family): key j (global position) is masked
                              for segment rows [lts_j, lte_j) U [uts_j, ute_j)            */
} lca_mask_kind;

typedef struct {
  int32_t q_off, q_len, k_off, k_len;
} lca_segment;

typedef struct {
  int32_t kind; /* lca_mask_kind */
  int32_t window_left, window_right; /* inclusive distances, >= 0 */
  int32_t num_global;                /* GLOBAL_SLIDING, >= 0 */
  int32_t prefix_len;                /* PREFIX_LM_CAUSAL, >= 0 */
  const int32_t* seg_prefix;         /* host [n_seg]: PREFIX_LM_DOC prefix per segment */
  int32_t block;                     /* CAUSAL_BLOCKWISE, BLOCK_CAUSAL_DOC, >= 1 */
  const int32_t* part_bounds;        /* host [n_part_bounds]: SHARED_QUESTION, strictly
                                        increasing key positions, part_bounds[0] == 0,
                                        last >= every segment's k_len, at most 64 */
  int32_t n_part_bounds;
  /* Block-sparse maps.  Block indices are over GLOBAL packed token positions
   * (query row q_off+i, key k_off+j); the mask is also limited to the segment. */
  int32_t q_block, kv_block;  /* UNIFORM: block sizes; kv_block >= 32            */
  const int32_t* qb_bounds;   /* VARIABLE host [n_qb+1]: 0 = b0 < b1 < ... , b_last >= Tq */
  const int32_t* kb_bounds;   /* VARIABLE host [n_kb+1]: every block but the last >= 32 */
  int32_t n_qb, n_kb;         /* VARIABLE: block counts (UNIFORM: ignored)         */
  int32_t heads_in_map;       /* 1 (one map for all heads) or Hq                   */
  const int32_t* blk_row_ptr; /* device [heads_in_map*n_qb+1]: CSR row starts      */
  const int32_t* blk_col_idx; /* device [blk_nnz]: kept kv block indices           */
  int64_t blk_nnz;
  /* FLASHMASK: device int32 [Tk][4] = {lts, lte, uts, ute} per global key
   * position, rows relative to the query segment reading that key; 16-byte
   * aligned.  One map for all heads. */
  const int32_t* col_bounds;
} lca_mask_desc;

typedef struct {
  int32_t Tq, Tk, Hq, Hkv, d;
  int32_t n_seg;
  const lca_segment* segs; /* host [n_seg] */
  float scale;             /* softmax scale; 0 selects 1/sqrt(d) */
} lca_shape;

/* Bytes of workspace that lca_attn_fwd (for_bwd = 0) or lca_attn_bwd
 * (for_bwd = 1) needs for this shape and mask; the same value serves
 * lca_mask_materialize and lca_mask_nnz.  Host only; no CUDA call. */
LCA_API lca_status lca_workspace_size(const lca_shape* shape, const lca_mask_desc* mask, int for_bwd, size_t* bytes);

/* Forward (FlashAttention-2 核心优化: Q-split work, deferred rescale, one LSE
 * per row).  q, k, v: device bf16 inputs; o: bf16 [Tq][Hq][d] output;
 * lse: float [Hq][Tq] output (outputs in device or mapped host memory).
 * q, k, v and o must be 16-byte aligned and lse 4-byte aligned
 * (LCA_ERR_INVALID_ARG otherwise); an o that is 32-byte aligned is written
 * with 32-byte stores, any other with 16-byte ones (same values). */
LCA_API lca_status lca_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const lca_shape* shape,
                        const lca_mask_desc* mask, void* workspace, size_t workspace_bytes, void* stream);

/* Backward (FlashAttention-2 核心优化, 反向传播: dK/dV per key tile, dQ in a
 * separate query-tile pass, D = rowsum(dO * O) prepass).  dout, q, k, v, o:
 * device bf16; lse: device float from lca_attn_fwd; dq, dk, dv: bf16 outputs
 * in device or mapped host memory (written, not accumulated).  Every bf16
 * pointer must be 16-byte aligned (LCA_ERR_INVALID_ARG otherwise); dq, and
 * dk with dv, are written with 32-byte stores when 32-byte aligned.
 * The dK/dV pass runs on a stream the library owns (one per device, highest
 * priority), forked from `stream` and joined back to it with events, so that
 * the dQ pass runs beside it; all of the call's work still comes after the
 * work queued on `stream` before the call and before the work queued after
 * it.  While a profiling hook is on (lca_set_kernel_events or
 * lca_set_cta_profile) the passes run one after another on `stream`. */
LCA_API lca_status lca_attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* o,
                        const float* lse, void* dq, void* dk, void* dv, const lca_shape* shape,
                        const lca_mask_desc* mask, void* workspace, size_t workspace_bytes, void* stream);

/* Attention dropout ("长上下文能力：FlashAttention vs. RingAttention",
 * FlashAttention-1 核心优化, 算子融合: dropout fused with the matmuls, the
 * mask and the softmax).  Inverted dropout on the probabilities:
 *     O = (P * Z / kp) V,  LSE that of P (unchanged by dropout),
 * with t = floor(256 p + 1/2) (at most 255) and kp = (256 - t) / 256.  Z_ij
 * for query head h, query row i (global packed index) and key j (counted
 * from the first key of row i's segment) is 1 iff byte j % 4 of word
 * (j % 16) / 4 of Philox4x32-10(counter = (j / 16, i, h, 0), key = (seed
 * low 32 bits, seed high 32 bits)) is >= t; the same Z is regenerated by the
 * backward, so a forward and a backward called with equal lca_dropout values
 * are consistent.  p must satisfy 0 <= p < 1 (LCA_ERR_INVALID_ARG
 * otherwise); t = 0 computes exactly what lca_attn_fwd / lca_attn_bwd do. */
typedef struct {
  float p;       /* drop probability */
  uint64_t seed; /* Philox key */
} lca_dropout;

/* lca_attn_fwd with dropout; dropout NULL means none. */
LCA_API lca_status lca_attn_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse,
                                const lca_shape* shape, const lca_mask_desc* mask, const lca_dropout* dropout,
                                void* workspace, size_t workspace_bytes, void* stream);
/* lca_attn_bwd with dropout: o and lse must come from lca_attn_fwd_dropout
 * with the same shape, mask and dropout values; dropout NULL means none. */
LCA_API lca_status lca_attn_bwd_dropout(const void* dout, const void* q, const void* k, const void* v,
                                const void* o, const float* lse, void* dq, void* dk, void* dv,
                                const lca_shape* shape, const lca_mask_desc* mask, const lca_dropout* dropout,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Merge of partial forward results ("长上下文能力：FlashAttention vs.
 * RingAttention", Blockwise Parallel Transformer and RingAttention sections:
 * attention over a union of disjoint key blocks is assembled from each
 * block's output and softmax normaliser).  Part p holds o_parts[p] (device
 * bf16 [Tq][Hq][d]) and lse_parts[p] (device float [Hq][Tq], natural log) for
 * the same queries over a key set disjoint from every other part's, e.g. one
 * lca_attn_fwd call per key chunk.  Writes
 *     lse[h][i] = log sum_p exp(lse_p[h][i])
 *     o[i][h]   = sum_p exp(lse_p[h][i] - lse[h][i]) * o_p[i][h]   (bf16)
 * and o = 0, lse = -inf for rows no part attends (every lse_p = -inf).
 * A causal mask split into key chunks is a FULL call for the chunks below the
 * diagonal plus a CAUSAL call whose segments pair each query chunk with its
 * own, equally long key chunk.
 * o_parts, lse_parts: HOST arrays of n_parts device pointers,
 * 1 <= n_parts <= LCA_MERGE_MAX_PARTS; o may alias o_parts[0] and lse
 * lse_parts[0].  d must be 128; o pointers 16-byte aligned, lse pointers
 * 4-byte aligned.  Asynchronous on `stream`; needs no workspace. */
#define LCA_MERGE_MAX_PARTS 16
LCA_API lca_status lca_attn_merge(const void* const* o_parts, const float* const* lse_parts, int32_t n_parts, void* o,
                                  float* lse, int32_t Tq, int32_t Hq, int32_t d, void* stream);

/* Core-attention disaggregation planner ("Efficient Long-context Language
 * Model Training by Core Attention Disaggregation": core attention is cut
 * into token-level tasks that attention servers rebatch to balance compute).
 * Host only; no CUDA call.  Cuts documents of lengths doc_len[0..n_docs) into
 * query shards and assigns them to n_servers so that the causal attention
 * work per server -- the cells (b(b+1) - a(a+1))/2 of each of its shards
 * [a, b) -- is balanced:
 *   1. each document is cut into equal pieces no longer than max_shard
 *      (0 = no limit; else max_shard >= 2 * min_shard);
 *   2. pieces go to the least-loaded server, most expensive first;
 *   3. while the most loaded server exceeds the mean by more than
 *      `tolerance` (relative), its most expensive piece at least 2*min_shard
 *      long is cut where its cells halve, and step 2 is redone.
 * Shard [a, b) of a document whose keys start at position s is the segment
 * {q_off: its place in the server's packed query buffer, q_len: b - a,
 *  k_off: s, k_len: b} of a CAUSAL call: it attends keys [s, s + b).
 * Shards come out ordered by server, then document, then start.  Up to
 * max_shards entries are written to `shards` (host) and the count to
 * n_shards; server_cells (host, n_servers entries, may be NULL) receives each
 * server's cells per head.  LCA_ERR_WORKSPACE if max_shards is too small
 * (n_shards then holds the count needed). */
typedef struct {
  int32_t doc;    /* document index                        */
  int32_t start;  /* first query token, document-relative  */
  int32_t len;    /* query tokens                          */
  int32_t server; /* attention server it is assigned to    */
} lca_cad_shard;
LCA_API lca_status lca_cad_plan(const int32_t* doc_len, int32_t n_docs, int32_t n_servers, int32_t min_shard,
                                int32_t max_shard, double tolerance, lca_cad_shard* shards, int32_t max_shards,
                                int32_t* n_shards, int64_t* server_cells);

/* ------------------------------------------------------------------ rotary positions
 * Between the projections and the attention kernels, the pairs of values of a
 * query's or key's head are turned by an angle that grows with its position,
 * so that scores depend on distances.  Pair i of a row at position p has the
 * angle p * inv_freq[i] and becomes
 *     scale * (a cos - b sin),  scale * (b cos + a sin)
 * Values at and behind rot_dim are copied.  inv_freq is read during the call;
 * the angle is found to 2^-32 of a turn at every position, cos, sin and the
 * products are 32-bit ones, and a result is rounded once. */
typedef struct {
  int32_t rot_dim;        /* values of a head that take part: even, 2 to d      */
  int32_t interleaved;    /* 0: pairs (i, i + rot_dim / 2); else (2 i, 2 i + 1) */
  const double* inv_freq; /* host [rot_dim / 2]: radians per position, 0 to 2^20 */
  float scale;            /* factor of the turned pairs, >= 0; 0 selects 1      */
} lca_rope_desc;

/* Rows of heads * d dense elements, strides apart (multiples of 8 elements, at
 * least heads * d).  y is written; y = x with the same stride turns in place.
 * q and k have fewer than 2^24 heads together (LCA_ERR_UNSUPPORTED). */
typedef struct {
  const void* x;
  void* y;
  int32_t heads;
  int64_t x_stride, y_stride;
} lca_rope_rows;

/* Turns row t of q and of k (either may be null) by positions[t] (int32,
 * device; negative ones turn the other way).  back != 0: by the opposite angle,
 * with the same scale, which takes the gradients of the results to those of
 * q and k.  dtype: lca_dtype of all rows; d must be 128; x and y 16-byte
 * aligned, device memory.  Rows written must not overlap positions or other
 * rows, but for x = y; rows of one stride that lie beside one another, as parts
 * of one projection, do not (LCA_ERR_INVALID_ARG otherwise). */
LCA_API lca_status lca_rope(const lca_rope_rows* q, const lca_rope_rows* k, const int32_t* positions, int32_t n_rows,
                            int32_t d, int32_t dtype, const lca_rope_desc* rope, int32_t back, void* stream);

/* Tables of frequencies.  With w_i = base^(-2 i / rot_dim), L = original_len:
 *   PLAIN   w_i
 *   LINEAR  w_i / factor (positions are interpolated)
 *   NTK     the same with base * factor^(rot_dim / (rot_dim - 2)) as the base
 *   YARN    blend of w_i and w_i / factor, linear in i between the pairs that
 *           make `fast` and `slow` turns in L positions (rounded down and up):
 *           the faster ones stay; scale = 0.1 ln(factor) + 1
 *   BANDS   blend of the same two, linear in the turns that pair i makes in L
 *           positions: at least `fast`, w_i stays; at most `slow`, w_i / factor
 * scale is 1 but for YARN.  base > 1, factor >= 1; YARN and BANDS need L >= 1
 * and 0 < slow < fast, NTK rot_dim > 2.  Host only; no CUDA call.
 * inv_freq: host [rot_dim / 2]. */
typedef enum {
  LCA_ROPE_PLAIN = 0,
  LCA_ROPE_LINEAR = 1,
  LCA_ROPE_NTK = 2,
  LCA_ROPE_YARN = 3,
  LCA_ROPE_BANDS = 4
} lca_rope_scaling;
typedef struct {
  int32_t rot_dim;
  int32_t scaling; /* lca_rope_scaling */
  double base, factor;
  int32_t original_len;
  double fast, slow;
} lca_rope_table;
LCA_API lca_status lca_rope_frequencies(const lca_rope_table* table, double* inv_freq, float* scale);

/* ------------------------------------------------------------------ paged cache
 * Serving: keys and values of earlier tokens live in pages of a cache, and a
 * batch of requests adds new tokens to it.  lca_paged_plan gives every new
 * token a place, lca_paged_write stores its key and value there, and
 * lca_attn_paged attends the new tokens to their requests' keys.  Lengths,
 * tables and page lists are read from device memory when the kernels run, so
 * a captured graph of the three calls serves later batches of the same shape.
 * A block table has one row per request: entry c is the page that holds the
 * request's tokens [c * page_size, (c + 1) * page_size). */
typedef enum { LCA_BF16 = 0, LCA_F16 = 1 } lca_dtype;

/* Token t of page p, KV head h starts at element
 *     p * page_stride + t * token_stride + h * head_stride
 * of k and of v (device or managed memory); its d elements are contiguous.
 * Any order of the axes is fine ([page][token][head] and
 * [page][head][token] among them, and K and V as parts of one array), as long
 * as the rows of k, and those of v, do not overlap.  Pages should be the
 * outermost axis: otherwise, and with more than 128 query heads per KV head,
 * lca_attn_paged serves prompts with the kernel made for single tokens, at
 * about a tenth of the speed.  Strides are multiples of
 * 8 elements, 8 to 2^38; k and v are 16-byte aligned; d must be 128.
 * page_size is a multiple of 8 (LCA_ERR_UNSUPPORTED otherwise) and
 * n_pages * page_size < 2^31. */
typedef struct {
  void* k;
  void* v;
  int32_t n_pages, page_size, Hkv, d;
  int32_t dtype; /* lca_dtype */
  int64_t page_stride, token_stride, head_stride;
} lca_paged_cache;

/* The batch's bookkeeping.  Request i has ctx_len[i] tokens in the cache and
 * new_len[i] new ones (0 allowed).  With have = ceil(ctx / page_size) and
 * want = ceil((ctx + new) / page_size), entries [have, want) of its table row
 * are filled with the next unused entries of free_pages, request after
 * request, starting at free_pages[taken[0]]; the other entries keep their
 * values.  Outputs (all int32, device):
 *   q_start [n_seq + 1]  first row of each request's new tokens, packed
 *   k_len [n_seq]        ctx + new
 *   slots [n_rows]       page * page_size + offset of each new token; -1 for
 *                        rows behind the last request
 *   positions [n_rows]   position of each new token in its request; 0 behind
 *   state [4]            {entries of free_pages used so far, pages that were
 *                        missing, requests whose lengths were unusable, new
 *                        tokens}
 * The call depends on nothing it writes, so it can be repeated.  Pass
 * state[0:1] of one call as `taken` of the next.  What cannot be served is
 * answered on the device, without a fault: an entry of free_pages outside
 * [0, n_pages) or past n_free becomes table entry -1, and a token on a page
 * outside [0, n_pages) gets slot -1; a negative length counts as 0; tokens
 * past max_pages * page_size get slot -1 and k_len stops there, but not
 * q_start; rows past n_rows are dropped: q_start stops there, but not k_len.
 * So where state[2] is not 0, the last q_len of k_len tokens need not be a
 * request's rows, and lca_attn_paged needs ctx_len as well (lca_paged_shape)
 * to place them.
 * ctx_len, new_len [n_seq], free_pages [n_free], taken [1]: int32, device.
 * block_table: int32, device, n_seq rows of max_pages entries, table_stride
 * entries apart (>= max_pages); n_seq below 2^30.  n_rows: rows of the packed batch, at least
 * the new tokens; 0 to 2^31 - 1.  Outputs must not overlap one another or an
 * input (LCA_ERR_INVALID_ARG). */
LCA_API lca_status lca_paged_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t n_seq,
                                  const int32_t* free_pages, int32_t n_free, const int32_t* taken,
                                  int32_t* block_table, int64_t table_stride, int32_t max_pages, int32_t page_size,
                                  int32_t n_pages, int32_t n_rows, int32_t* q_start, int32_t* k_len, int32_t* slots,
                                  int32_t* positions, int32_t* state, void* stream);

/* Stores row r of k and v (device, the cache's dtype, Hkv heads of d dense
 * elements, rows k_stride and v_stride elements apart) as token
 * slots[r] % page_size of page slots[r] / page_size.  A row whose slot lies
 * outside [0, n_pages * page_size) is skipped (padding rows have -1); the
 * slots of the other rows must differ (of two rows with one slot, either may
 * be stored, or parts of both).  Row strides are multiples of 8 elements and
 * k, v 16-byte aligned; k, v and slots must not overlap the cache
 * (LCA_ERR_INVALID_ARG; it counts from its first to its last element). */
LCA_API lca_status lca_paged_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                   const int32_t* slots, int32_t n_rows, const lca_paged_cache* cache, void* stream);

typedef struct {
  int32_t Tq, Hq, n_seq;
  int32_t max_pages;    /* entries of a table row                            */
  int64_t table_stride; /* entries between table rows, >= max_pages          */
  int64_t q_stride;     /* elements between rows of q, >= Hq * d, multiple of 8 */
  int32_t max_q_len;    /* no request has more new tokens than this; 0: not
                           known.  Chooses kernels, never results.  A decode
                           step that gives 1 needs 26 MB of workspace and two
                           launches, not 94 and four.                        */
  float scale;          /* softmax scale; 0 selects 1/sqrt(d)                */
  const int32_t* ctx_len; /* null, or device int32 [n_seq]: the tokens that
                           each request had before its new ones, as given to
                           lca_paged_plan                                    */
} lca_paged_shape;

/* Attention of new tokens over the cache: row q_start[i] + t of q is new
 * token t of request i, at position ie = t + k_len[i] - (q_start[i + 1] -
 * q_start[i]) of its k_len[i] tokens, and attends those keys that the mask
 * keeps (positions as in lca_mask_kind, the request being the segment; the
 * new tokens' own keys must be in the cache already).  A request with one new
 * token is a decode step, one with many a prompt or a chunk of one; a batch
 * may mix them.
 * With shape->ctx_len new token t is at position ie = t + ctx_len[i] whatever
 * k_len[i] is, and its request has no keys past the last of its rows: the
 * same where k_len[i] = ctx_len[i] + new tokens, and right also where
 * lca_paged_plan had no room for some of them.  A token at or past k_len[i]
 * has no key and attends nothing.
 * Masks: FULL, CAUSAL, SLIDING, CAUSAL_SLIDING, DOC,
 * CAUSAL_DOC, GLOBAL_SLIDING, CAUSAL_BLOCKWISE, PREFIX_LM_CAUSAL and
 * BLOCK_CAUSAL_DOC (LCA_ERR_UNSUPPORTED for the others).
 * q: device, the cache's dtype, [Tq] rows of Hq * d dense elements, q_stride
 * apart, 16-byte aligned.  block_table: int32, device.  q_start: int32
 * [n_seq + 1], k_len: int32 [n_seq], device.  o: [Tq][Hq][d] dense, the
 * cache's dtype, 16-byte aligned; lse: float [Hq][Tq], natural log, as
 * lca_attn_fwd writes it and lca_attn_merge reads it (whose o parts are bf16).
 * The weights are rounded to the cache's dtype before their product with V;
 * in fp16 one below 2^-31 of the row's largest may count as 0.  o, lse and the
 * workspace must not overlap one another or an input (LCA_ERR_INVALID_ARG;
 * the cache counts from its first to its last element).  Rows that attend
 * nothing, and rows outside every request, get o = 0, lse = -inf.
 * Nothing that lies in the cache behind a request's last key, or in keys
 * that the mask hides from all of its new tokens, reaches a result (infinities
 * and NaN included).  An infinity or NaN in the values of a key makes that
 * element of o infinite or NaN in the rows that attend the key, and in no
 * other (NaN also for an infinity whose weight rounds to 0).  GLOBAL_SLIDING's
 * first num_global tokens attend all keys that are there, so a prompt taken in
 * chunks gives them other results than one taken at once.  A table entry outside [0, n_pages) that a row needs
 * reads as zeros; q_start that decreases or leaves [0, Tq] and k_len or
 * ctx_len outside [0, max_pages * page_size] are clamped; each, and a token at
 * or past k_len[i] where ctx_len is given, sets LCA_ERR_DEVICE_ARG in the
 * status word (lca_read_status). */
LCA_API lca_status lca_attn_paged(const void* q, const lca_paged_cache* cache, const int32_t* block_table,
                                  const int32_t* q_start, const int32_t* k_len, void* o, float* lse,
                                  const lca_paged_shape* shape, const lca_mask_desc* mask, void* workspace,
                                  size_t workspace_bytes, void* stream);
/* Bytes of workspace that lca_attn_paged needs (256-byte aligned).  Host
 * only; no CUDA call.  Two calls that may run at once need a workspace each. */
LCA_API lca_status lca_attn_paged_workspace_size(const lca_paged_shape* shape, const lca_paged_cache* cache,
                                                 const lca_mask_desc* mask, size_t* bytes);

/* ------------------------------------------------------------------ paged cache of 8 bits
 * A paged cache whose rows (a token's d values of one KV head) are e4m3 values
 * times a power of two: value = e4m3 * 2^(b - 127), with a byte b per row.  It
 * holds half the bytes of a 16-bit cache, which is what generation is bound by.
 * Each value is off by at most 2^-4 of itself (half a step of its 3 bits), or
 * by 2^-10 * 2^(b - 127) where that is more.  Bytes count as the nearest one of
 * LCA_FP8_SCALE_MIN to LCA_FP8_SCALE_MAX.
 * Token t of page p, head h: d bytes at p * page_stride + t * token_stride +
 * h * head_stride of k and of v, and a byte at p * scale_page_stride + h *
 * scale_head_stride + t of k_scale and of v_scale.  Strides of values are
 * multiples of 16, those of scales of 8, all 8 to 2^38; k and v are
 * 16-byte, the scales 8-byte aligned; Hkv is below 2^24 (LCA_ERR_UNSUPPORTED).
 * Otherwise as lca_paged_cache, whose lca_paged_plan serves both. */
#define LCA_FP8_SCALE_MIN 79  /* 2^-48 */
#define LCA_FP8_SCALE_MAX 175 /* 2^48 */
typedef struct {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int32_t n_pages, page_size, Hkv, d;
  int64_t page_stride, token_stride, head_stride;
  int64_t scale_page_stride, scale_head_stride;
} lca_paged_cache_fp8;

/* lca_paged_write into such a cache: k and v (device, dtype's elements) are
 * quantised as they are stored.  b is the smallest byte for which the row's
 * largest finite magnitude is at most 448 * 2^(b - 127); values are divided by
 * 2^(b - 127), which is exact, and rounded to the nearest e4m3 value, the even
 * one of two.  Magnitudes past 448 * 2^48 become that; infinities and NaN are
 * stored as NaN.  Slots, alignment and overlaps as lca_paged_write (the cache
 * counts with its scales). */
LCA_API lca_status lca_paged_write_fp8(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int32_t dtype,
                                       const int32_t* slots, int32_t n_rows, const lca_paged_cache_fp8* cache,
                                       void* stream);

/* Reads pages back: page i of `out` gets the 16-bit form of page pages[i] of
 * `cache`, all of its tokens and heads, K and V.  A product of an e4m3 value
 * and a power of two is exact in bf16; in fp16 what lies outside its range is
 * rounded, beyond 65504 to that.  out: page_size, Hkv and d as the cache's, n_pages
 * at least n.  An entry outside [0, cache->n_pages) leaves its page of out
 * as it was, so the block tables of a batch, flattened, are a list of pages,
 * and out is their cache for lca_attn_paged with the table 0, 1, 2, ...; an
 * out of token stride Hkv * d, head stride d is rows of packed keys for
 * lca_attn_fwd (which multiplies what lies behind a segment's last key by 0:
 * slots that were never written must hold no NaN for it).  pages: int32,
 * device.  out must not overlap the cache or pages (LCA_ERR_INVALID_ARG).
 * page_size * Hkv is below 2^31 - 256 (LCA_ERR_UNSUPPORTED). */
LCA_API lca_status lca_paged_read_fp8(const lca_paged_cache_fp8* cache, const int32_t* pages, int32_t n,
                                      const lca_paged_cache* out, void* stream);

/* lca_attn_paged over such a cache: the same arguments, masks, reports and
 * rules, with q and o of the given lca_dtype; Hq is below 2^24.  Scores are those
 * of the values that the cache stands for; values of q below 2^-28 of the largest
 * of their row (a token's d values of one head) may lose bits.  A request's new
 * tokens times Hq / Hkv are its rows per KV head, and how weights are rounded
 * before their product with V depends on them and on the batch:
 *  * where no request can have more than 32 (max_q_len, or Tq), and in other
 *    batches for those of at most 16: to 11 bits times their key's factor; a key
 *    whose weight times factor is below 2^-36 of the row's largest may count as 0.
 *  * otherwise likewise, with 2^-24; and where factors of 32 keys that lie together
 *    are below 2^-22 (K) or 2^-8 (V) of the largest among 128, these 128 keys take
 *    about twice the time.
 *  * instead of that, where q is bf16, requests have 1536 rows and more on average
 *    (max_q_len or Tq / n_seq), Hq / Hkv is 128 at most, and the tables' entries,
 *    all of them, are 1 GiB as 16-bit K and V at most: the pages that those rows
 *    attend are read back (lca_paged_read_fp8, exact in bf16) into the workspace
 *    first, and weights are rounded to bf16, ones below 2^-126 of the row's
 *    largest to 0.  A workspace may so need up to 1 GiB more.
 * NaN in the values of a key as in lca_attn_paged. */
LCA_API lca_status lca_attn_paged_fp8(const void* q, int32_t dtype, const lca_paged_cache_fp8* cache,
                                      const int32_t* block_table, const int32_t* q_start, const int32_t* k_len, void* o,
                                      float* lse, const lca_paged_shape* shape, const lca_mask_desc* mask,
                                      void* workspace, size_t workspace_bytes, void* stream);
/* As lca_attn_paged_workspace_size.  What max_q_len = 0 needs serves every other,
 * and queries of both types are served (fp16 ones need no room for a copy). */
LCA_API lca_status lca_attn_paged_fp8_workspace_size(const lca_paged_shape* shape, const lca_paged_cache_fp8* cache,
                                                     const lca_mask_desc* mask, size_t* bytes);

/* Test hook: writes the mask of one segment and query head, evaluated by the
 * same device predicate the attention kernels apply, as bytes (1 = attend)
 * into `out` (device, q_len*k_len, row-major). */
LCA_API lca_status lca_mask_materialize(const lca_shape* shape, const lca_mask_desc* mask, int32_t head, int32_t seg,
                                uint8_t* out, void* workspace, size_t workspace_bytes, void* stream);

/* Test hook: the tile classes of one segment and query head for 128 x 128
 * tiles, one byte per tile written to `out` (device, nq*nk bytes, row-major,
 * nq = ceil(q_len/128), nk = ceil(k_len/128)).  Bits 0-1: 0 empty, 1 full,
 * 2 partial.  A partial tile also sets bit 2 when its query rows [0, 64)
 * attend no key of the tile, bit 3 when its rows [64, 128) (those inside the
 * segment) attend none; the backward key-gradient pass skips those halves. */
LCA_API lca_status lca_mask_tile_classes(const lca_shape* shape, const lca_mask_desc* mask, int32_t head, int32_t seg,
                                 uint8_t* out, void* workspace, size_t workspace_bytes, void* stream);

/* Number of attended (query, key) cells per query head, summed over
 * segments, written to `nnz` (device, uint64 [Hq]).  Used for the effective
 * FLOP count 4*d*nnz (forward) and 10*d*nnz (backward). */
LCA_API lca_status lca_mask_nnz(const lca_shape* shape, const lca_mask_desc* mask, uint64_t* nnz, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Forward pass with a library-owned workspace, for callers that cannot
 * allocate device memory: processes whose device-memory pool was carved out
 * up front and may not grow, or code running where an allocation is not
 * allowed (inside an allocator's own callback, for example).  The pages have
 * no counterpart: this is a deployment convenience of this library.
 * Arguments and results are those of lca_attn_fwd; the caller still passes
 * (and owns) q, k, v, o and lse.
 * Scratch: one static device array of LCA_STATIC_WORKSPACE_BYTES (16 MiB),
 * which every GPU that loads this library holds until the process exits.  A
 * shape whose forward workspace (lca_workspace_size with for_bwd = 0) is
 * larger is rejected with LCA_ERR_WORKSPACE before anything is launched, and
 * lca_last_error_detail says how much it needed.
 * The array is reserved on a device when CUDA loads this library's device
 * code there: with CUDA's default lazy loading that happens at the latest
 * during the first call of this function on the device, which can then fail
 * with LCA_ERR_CUDA if the device is already full.  Make that first call at
 * set-up time, before the rest of device memory is handed out (a small shape
 * will do); it also looks up the array's device address with that device
 * current, so it must come before any stream capture.
 * Every call on a device shares the one array and clears what must start at
 * zero; calls that overlap on the GPU (two streams, or two host threads)
 * race on it, so the caller must serialise them.
 * No device memory is allocated: no cudaMalloc, cudaFree or allocating
 * library routine is called. */
#define LCA_STATIC_WORKSPACE_BYTES (16u << 20)
LCA_API lca_status lca_attn_fwd_static_workspace(const void* q, const void* k, const void* v, void* o, float* lse,
                                                 const lca_shape* shape, const lca_mask_desc* mask, void* stream);

/* Synchronises `stream`, then copies the device status word of the last
 * call that used this workspace: out[0] = lca_status code (0 = none),
 * out[1] = where it was raised.  Each fwd/bwd call clears it first. */
LCA_API lca_status lca_read_status(const void* workspace, int32_t out[2], void* stream);

/* Test hook: launches one block that waits on a barrier nothing arrives at,
 * with a wait limit of `limit_ms`; it must record LCA_ERR_TIMEOUT in the
 * workspace status word and exit. */
LCA_API lca_status lca_probe_wait_timeout(void* workspace, size_t workspace_bytes, int32_t limit_ms, void* stream);

/* Profiling hook.  With a non-null ring of CUDA events (cudaEvent_t handles
 * passed as void*, n_events even), every later fwd/bwd call records one
 * event pair around each of its phases, on its own stream, taking the next
 * pair of the ring (the cursor restarts at each call of this function):
 *   lca_attn_fwd: 0 = mask compiler + cost sort, 1 = forward kernel
 *   lca_attn_bwd: 2 = D prepass, 3 = dK/dV lists + sort, 4 = dK/dV kernel,
 *                 5 = dQ lists + sort, 6 = dQ kernel
 * The phase of each recorded pair is written to `phases` (host, n_events/2
 * entries, may be null).  Pass null to stop.  Process-wide, not thread-safe. */
LCA_API lca_status lca_set_kernel_events(void* const* events, int32_t n_events, int32_t* phases);

/* Profiling hook: per-CTA work and time of the attention kernels, the
 * evidence for how evenly the cost-sorted persistent scheduler spreads work
 * over the SMs.  With a non-null device buffer `buf` of at least
 * LCA_CTA_PROFILE_BYTES (8-byte aligned), every later forward and backward
 * call writes one record per CTA of each attention kernel it launches:
 * kernel slot k (0 forward, 1 dK/dV, 2 dQ) starts at byte k * 1024 * 64, and
 * CTA b's record at 64 * b within it, eight uint64 values:
 *   start and end of the CTA (%globaltimer, ns), work items it ran, full and
 *   partial tile units it ran (forward: 128-row query sub-tile x key tile;
 *   dK/dV: 64-row query step; dQ: 128-row query tile x key tile), the grid
 *   size, the SM it ran on, 0.
 * A call clears its kernel's slot on its stream before the launch, so
 * records of CTAs beyond the grid are zero.  Pass null to stop.
 * LCA_ERR_INVALID_ARG for a short, misaligned or non-device buffer.
 * Process-wide, not thread-safe. */
#define LCA_CTA_PROFILE_BYTES (3u * 1024u * 64u)
LCA_API lca_status lca_set_cta_profile(void* buf, size_t bytes);

/* Text of the last CUDA failure seen by this library in the calling thread
 * (the failing call and the runtime's message), or "" if none. */
LCA_API const char* lca_last_error_detail(void);

/* Number of kernels this library has launched since it was loaded. */
LCA_API uint64_t lca_launch_count(void);

LCA_API const char* lca_status_string(lca_status status);
/* Library revision, 100 + n; n grows whenever an entry point's behaviour
 * changes (102: lca_mask_tile_classes reports the empty-half flags; 103:
 * outputs may be mapped host memory, and every pointer's kind is checked;
 * 104: device pointers of another device than the current one are refused;
 * 105: the paged cache; 106: lca_paged_shape.ctx_len; 107: rotary positions and
 * the paged cache of 8 bits). */
LCA_API int32_t lca_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LCA_ATTN_H */
