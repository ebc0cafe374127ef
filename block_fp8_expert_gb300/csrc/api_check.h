// Argument checks and error returns shared by the files that implement the C
// ABI.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "moe_internal.h"

namespace moe {

// Records the formatted text for moe_last_error_message() and returns s.
inline moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

inline moe_status cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();  // reported here: the caller's next CUDA check shall not meet it again
  return fail(MOE_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline size_t align_up(size_t v) { return (v + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace moe

#define REQUIRE_PTR(p)                                                                    \
  do {                                                                                    \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);               \
    if (!aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

#define REQUIRE_OPT_PTR(p)                                                   \
  do {                                                                       \
    if ((p) != nullptr && !aligned16(p))                                     \
      return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p);    \
  } while (0)

// For arrays that are read or written one element at a time.
#define REQUIRE_ELEMENTS(p)                                                                 \
  do {                                                                                      \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);                 \
    if (reinterpret_cast<uintptr_t>(p) % sizeof(*(p)))                                      \
      return fail(MOE_ERR_INVALID_ARG, "%s is not aligned to its %zu-byte elements", #p,    \
                  sizeof(*(p)));                                                            \
  } while (0)

#define CUDA_CHECK(expr, where)                           \
  do {                                                    \
    cudaError_t e_ = (expr);                              \
    if (e_ != cudaSuccess) return cuda_fail(e_, where);   \
  } while (0)
