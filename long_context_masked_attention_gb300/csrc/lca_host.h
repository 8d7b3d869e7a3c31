// lca_host.h — host helpers shared by the files that implement the C ABI:
// error text, pointer checks, device properties.  Defined in lca_api.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

#include "../../include/lca_attn.h"

namespace lca {

constexpr size_t kAlign = 256;  // workspace and its parts
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Record the text that lca_last_error_detail returns; both give LCA_ERR_CUDA.
lca_status cuda_fail(const char* what, cudaError_t e);
lca_status driver_fail(const char* what, int code);

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // null where the driver lacks it
int num_sms();                                  // of the current device; 0 (with error text) on failure
unsigned long long wait_limit_ns();

bool device_input(const void* p);
void* output_address(void* p);

}  // namespace lca

#define LCA_CUDA(x)                                       \
  do {                                                    \
    const cudaError_t e_ = (x);                           \
    if (e_ != cudaSuccess) return lca::cuda_fail(#x, e_); \
  } while (0)
