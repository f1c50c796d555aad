// plan.hpp -- lists of tensors that one launch takes in chunks: which tensor a chunk is of, and
// whether tensors share memory (internal; AdamW and the gradients' norm share it).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

namespace grpo {

// The last tensor whose first chunk is <= chunk: a 64-way search, one load per level.
// (A tensor of no elements has the first chunk of the next one and is never the last.)
__device__ __forceinline__ int owner_of(const int64_t* __restrict__ first, int count,
                                        int64_t chunk) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = count;
  while (len > 1) {
    const int stride = (len + 63) / 64;
    const bool le = lane * stride < len && first[lo + lane * stride] <= chunk;
    const int k = __popcll(__ballot(le)) - 1;
    lo += k * stride;
    len = min(stride, len - k * stride);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

struct Range {
  uintptr_t from, to;
  bool written;
};

// Two ranges that share a byte, one of them written, would race.
inline bool any_overlap(std::vector<Range>& r) {
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  uintptr_t read_end = 0, write_end = 0;
  for (const Range& x : r) {
    if (x.from < write_end || (x.written && x.from < read_end)) return true;
    (x.written ? write_end : read_end) = std::max(x.written ? write_end : read_end, x.to);
  }
  return false;
}

constexpr int64_t kMaxTensors = 1 << 24;
constexpr int64_t kMaxBlocks = (1 << 24) - 1;   // a grid of 256-thread blocks stays below 2^32 threads

}  // namespace grpo
