// lca_paged8_chunk.cu — attention of many rows over an 8-bit paged cache
// (lca_paged_chunk.cuh).
#include "lca_paged_chunk.cuh"

namespace lca {

cudaError_t launch_paged_chunk8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedAttnArgs& a, bool fp16, int num_sms, cudaStream_t st) {
  return fp16 ? launch_chunk<__half, true>(tq, tk, tv, a, num_sms, st)
              : launch_chunk<__nv_bfloat16, true>(tq, tk, tv, a, num_sms, st);
}

}  // namespace lca
