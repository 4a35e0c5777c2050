// Argument checks of the C entry points outside gdn_abi.cu: host code only.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "gdn_internal.h"

namespace gdn {

inline gdn_status_t failf(gdn_status_t st, const char *fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_host_error(st, msg);
}

inline bool aligned_to(const void *p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// The status of a launch; the runtime's last-error slot is emptied, since the
// status carries the error.
inline gdn_status_t launch_status(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return GDN_OK;
  (void)cudaGetLastError();
  return failf(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline size_t dtype_bytes(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// SMs of the current device, read once for each (a GB300's count if it cannot
// be read).
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 152;
  }
  n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return 152;
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Tokens of a batch row, or rows of a head: the kernels' indexes run up to 256 past the last one.
constexpr int MAX_TOKENS = 0x7fffff00;

#define CHECK_THAT(cond, st, ...)                       \
  do {                                                  \
    if (!(cond)) return ::gdn::failf(st, __VA_ARGS__);  \
  } while (0)

#define CHECK_OPT_PTR(ptr, name)                                                        \
  CHECK_THAT((ptr) == nullptr || ::gdn::aligned_to(ptr, 16), GDN_ERR_MISALIGNED,        \
             "%s is not 16-byte aligned", name)

#define CHECK_PTR(ptr, name)                                                            \
  do {                                                                                  \
    CHECK_THAT((ptr) != nullptr, GDN_ERR_INVALID_ARG, "%s must not be NULL", name);     \
    CHECK_OPT_PTR(ptr, name);                                                           \
  } while (0)

// Token tensors may start at any element: column ranges of wider buffers do.
#define CHECK_TOKENS(ptr, name, dtype)                                                  \
  do {                                                                                  \
    CHECK_THAT((ptr) != nullptr, GDN_ERR_INVALID_ARG, "%s must not be NULL", name);     \
    CHECK_THAT(::gdn::aligned_to(ptr, ::gdn::dtype_bytes(dtype)), GDN_ERR_MISALIGNED,   \
               "%s is not aligned to its type", name);                                  \
  } while (0)

#define CHECK_DTYPE(dt, name)                                                           \
  CHECK_THAT((dt) == GDN_F32 || (dt) == GDN_BF16, GDN_ERR_INVALID_ARG,                  \
             "%s %d is not GDN_F32/GDN_BF16", name, (int)(dt))

#define CHECK_FLAG(v, name) \
  CHECK_THAT((v) == 0 || (v) == 1, GDN_ERR_INVALID_ARG, "%s must be 0 or 1", name)

}  // namespace gdn
