// api.hpp -- what the files that define C-ABI entry points share: the error text, the
// workspace alignment and the checks of pointers and HIP calls (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/grpo.h"

namespace grpo {

// Sets this thread's error text (grpo_last_error) and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* where);
void clear_error();
const char* last_error();

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// Memory that a call reads or writes (null: none).  Blocks write while others still read, so what is
// written has to lie apart from what is read and from what else is written: whether it does.
struct Memory {
  const void* at;
  size_t bytes;
};
inline bool share(const Memory& a, const Memory& b) {
  return a.at != nullptr && b.at != nullptr && (uintptr_t)a.at < (uintptr_t)b.at + b.bytes &&
         (uintptr_t)b.at < (uintptr_t)a.at + a.bytes;
}
inline bool apart(std::initializer_list<Memory> written, std::initializer_list<Memory> read) {
  for (const Memory* w = written.begin(); w != written.end(); ++w) {
    for (const Memory* o = w + 1; o != written.end(); ++o)
      if (share(*w, *o)) return false;
    for (const Memory& r : read)
      if (share(*w, r)) return false;
  }
  return true;
}

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
