// lca_paged.h — what the paged-cache entry points (lca_paged_api.cu) and
// their kernels share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "lca_common.cuh"

namespace lca {

void note_launches(int n);

struct PagedPlanArgs {
  const int *ctx_len, *new_len, *free_pages, *taken;
  int* block_table;
  long long table_stride;
  int n_seq, n_free, max_pages, page_size, n_pages, n_rows;
  int *q_start, *k_len, *slots, *positions, *state;
};
void launch_paged_plan(const PagedPlanArgs& a, int num_sms, cudaStream_t st);

// Strides in 16-byte units.
struct PagedWriteArgs {
  const uint4 *k, *v;
  uint4 *kc, *vc;
  long long k_stride, v_stride, page_stride, token_stride, head_stride;
  const int* slots;
  int n_rows, Hkv, page_size, n_slots;
};
void launch_paged_write(const PagedWriteArgs& a, int num_sms, cudaStream_t st);

// Attention over few rows: at most this many CTAs and spans of work, each span
// with two workspace slots for unfinished sums (16 rows of O, maximum, sum).
constexpr int kPagedMaxCtas = 512;
constexpr int kPagedMaxSpans = 3 * kPagedMaxCtas;
constexpr int kPagedPartFloats = 16 * (kHeadDim + 2);
// Over many rows: the same with 256 rows.
constexpr int kPagedMaxChunkCtas = 256;
constexpr int kPagedChunkPartFloats = 256 * (kHeadDim + 2);
// Requests with up to this many rows (new tokens x query heads of a group)
// per KV head go to the kernel for few rows when both kernels run.  16 is one
// tile of it; with 32, in two tiles that read the keys twice, 32 requests of
// 3-4 tokens at 1K-16K keys, 64 heads on 8, take 335 us where padded tiles of
// 128 rows take 202; 32 of a token at 1K-8K with one group of 24 heads take 35
// either way.
constexpr int kPagedFewRows = 16;

// An item of many rows that goes on past the span of the CTA it starts in.
struct alignas(32) PagedCut {
  int last;  // CTA of its last piece, -1: no such item
  int late;  // its first piece is not the first of its CTA's span
  int head, tok0, q_off, q_len, pad[2];
};

struct PagedAttnArgs {
  MaskCtx mask;
  const void* q;
  const void *kc, *vc;
  long long q_stride, page_stride, token_stride, head_stride, table_stride;  // elements
  const uint8_t *ks, *vs;  // an 8-bit cache's factors, a byte per row
  long long scale_page_stride, scale_head_stride;
  const int *table, *q_start, *k_len;
  const int* ctx_len;  // null: a request's rows are the last of its k_len tokens
  void* o;
  float* lse;
  int* status;
  int* arrived;  // [kPagedMaxSpans] pieces finished of the split item that starts in a span
  int* claims;   // [1] spans claimed past the CTAs' first ones
  float* parts;  // [kPagedMaxSpans][2][rows of an item x (kHeadDim + 2)]
  int Tq, Hq, Hkv, G, n_seq, max_pages, page_size, n_pages;
  uint32_t page_mul;  // page_divisor's
  int page_shift;
  float scale_log2;
  int few;  // rows per KV head up to which the kernel for few rows serves a request
  // the kernel for many rows
  int tpt;       // tokens of a 128-row sub-tile: floor(128 / G)
  int box_rows;  // keys of one TMA box: gcd(page_size, 128)
  bool head_first;  // the K and V maps' axes: 64 values, head, token, page; else token before head
  int max_blocks;
  int* block0;        // [n_seq + 1] row blocks before each request
  long long* line;    // [max_blocks + 1] key tiles before each row block
  float* chunk_parts; // [kPagedMaxChunkCtas][2][kPagedChunkPartFloats]
  PagedCut* cuts;     // [kPagedMaxChunkCtas], by the CTA it starts in
  int out_v8;         // o is 32-byte aligned
  unsigned long long wait_limit_ns;
};
// A call is begin and decode or, where some request may have many rows,
// begin, chunk, decode (behind), join.  Each later kernel is launched while
// the one before it runs.
cudaError_t launch_paged_begin(const PagedAttnArgs& a, bool many, cudaStream_t st);
cudaError_t launch_paged_decode(const PagedAttnArgs& a, bool behind, bool fp16, int num_sms, cudaStream_t st);
// Queries as boxes of tpt tokens x G heads x 64, keys and values as boxes of
// box_rows tokens of one page and head x 64, 128-byte swizzled.
cudaError_t launch_paged_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st);
cudaError_t launch_paged_join(const PagedAttnArgs& a, bool fp16, bool eight, int num_sms, cudaStream_t st);

// Lets `kernel` use `bytes` of dynamic shared memory on the current device;
// asks CUDA once per device.  One `done` per kernel, bit d for device d.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches `kernel` so that it may start before the kernel in front of it on
// `st` has ended (it calls grid_wait before it touches what that one wrote).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace lca
