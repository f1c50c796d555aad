// elem.hpp -- rows of f32 or bf16 elements as 16-byte vectors at any element alignment,
// and sums over the lanes of a row (internal; the memory-bound operators share it).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace grpo {

// 16 bytes of elements, aligned to one element only: gfx950 loads and stores dwords at any
// byte address, so a row that starts at an odd element takes the same instruction as an
// aligned one.
template <typename T> struct Vec16;
template <> struct Vec16<float> {
  typedef __attribute__((ext_vector_type(4), aligned(4))) float type;
};
template <> struct Vec16<__bf16> {
  typedef __attribute__((ext_vector_type(8), aligned(2))) __bf16 type;
};
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// Elements [c, c + kVec) of a row of n; those at n and behind it read as zero.
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type load_vec(const T* row, int64_t c, int64_t n) {
  typedef typename Vec16<T>::type V;
  if (c + kVec<T> <= n) return *(const V*)(row + c);
  V v = {};
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j)
    if (c + j < n) v[j] = row[c + j];
  return v;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int64_t c, int64_t n, typename Vec16<T>::type v) {
  typedef typename Vec16<T>::type V;
  if (c + kVec<T> <= n) {
    *(V*)(row + c) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j)
    if (c + j < n) row[c + j] = v[j];
}

}  // namespace grpo
