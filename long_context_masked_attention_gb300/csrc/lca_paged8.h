// lca_paged8.h — what the entry points of the 8-bit paged cache
// (lca_paged_api.cu) and their kernels share.
#pragma once
#include "lca_paged.h"

namespace lca {

// Rows' factors are 2^-48 to 2^48: with weights of exponent at least -126
// (fp32's normal numbers) two keys of the same weight may have factors that far
// apart and both count, whichever of them the running maximum goes by.
constexpr int kScaleBias = 127;
constexpr int kScaleMin = -48, kScaleMax = 48;

// Strides of rows in elements, of the cache in bytes.
struct PagedWrite8Args {
  const uint16_t *k, *v;
  uint8_t *kc, *vc, *ks, *vs;
  long long k_stride, v_stride, page_stride, token_stride, head_stride, scale_page_stride, scale_head_stride;
  const int* slots;
  int n_rows, Hkv, page_size, n_slots;
  bool in_v8;  // every 16 values of k and v start on a 32-byte boundary
};
void launch_paged_write8(const PagedWrite8Args& a, bool fp16, int num_sms, cudaStream_t st);

struct PagedRead8Args {
  const uint8_t *kc, *vc, *ks, *vs;
  uint16_t *k, *v;
  long long page_stride, token_stride, head_stride, scale_page_stride, scale_head_stride;
  long long out_page_stride, out_token_stride, out_head_stride;
  const int* pages;
  int n, n_pages, Hkv, page_size;
  bool token_first;  // tokens of a head lie closer together than its heads
  bool out_v8;       // every 16 values of the result start on a 32-byte boundary
};
void launch_paged_read8(const PagedRead8Args& a, bool fp16, int num_sms, cudaStream_t st);

// The maps of K and V have boxes of box_rows rows of 128 bytes.
cudaError_t launch_paged_chunk8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st);
// The pages that the batch m needs, of its tables, n = n_seq max_pages; map: its
// tables over the copy.
void launch_paged_copy8(const PagedRead8Args& a, const PagedAttnArgs& m, int* map, bool fp16, int num_sms, cudaStream_t st);

// Attention over few rows, in items of `rows` of them, a multiple of 8.
// Where no request has more than these, the call needs no kernel for many rows.
constexpr int kPaged8FewRows = 32;
cudaError_t launch_paged_decode8(const PagedAttnArgs& a, int rows, bool behind, bool fp16, int num_sms, cudaStream_t st);

}  // namespace lca
