// api.hpp -- what the files that define C-ABI entry points share: the error text, the
// workspace alignment and the checks of pointers and HIP calls (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/grpo.h"

namespace grpo {

// Sets this thread's error text (grpo_last_error) and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* where);
void clear_error();
const char* last_error();

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

}  // namespace grpo

#define GRPO_CHECK_PTR(p)                                                          \
  do {                                                                             \
    if ((p) == nullptr) return grpo::fail(GRPO_ERR_INVALID_ARG, "null pointer: %s", #p); \
  } while (0)

#define GRPO_HIP(call)                                    \
  do {                                                    \
    hipError_t e_ = (call);                               \
    if (e_ != hipSuccess) return grpo::hip_fail(e_, #call);     \
  } while (0)
