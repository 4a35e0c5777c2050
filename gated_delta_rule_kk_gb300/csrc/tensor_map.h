// The CUDA driver's tensor map encoder, for the host code of kernels that load by TMA.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

namespace gdn {

// Looked up once (NULL if the driver has none); calls may come from several threads.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  auto fn = known.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      known.store(fn, std::memory_order_relaxed);
    }
  }
  return fn;
}

}  // namespace gdn
