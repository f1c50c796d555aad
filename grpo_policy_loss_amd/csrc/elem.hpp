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

// Elements [c, c + kVec) of a row of n; those at n and behind it read as zero.  In two steps: the
// load, which takes the row's last kVec elements where the asked ones pass the end, and what
// shifts them into place once they have arrived.  (Loading under a branch would make a wave that
// the row's end falls into wait for each load before the next.)
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type fetch_vec(const T* row, int c, int n) {
  typedef typename Vec16<T>::type V;
  if (n >= kVec<T>) return *(const V*)(row + min(c, n - kVec<T>));
  V v = {};
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j)
    if (c + j < n) v[j] = row[c + j];
  return v;
}
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type place_vec(typename Vec16<T>::type v, int c, int n) {
  const int over = c + kVec<T> - n;    // elements that are not the row's
  if (over <= 0 || n < kVec<T>) return v;
  typedef __attribute__((ext_vector_type(2))) uint64_t U2;
  U2 u = __builtin_bit_cast(U2, v);
  const int bits = over * 8 * (int)sizeof(T);
  if (bits >= 128) u = U2{0, 0};
  else if (bits >= 64) u = U2{u[1] >> (bits - 64), 0};
  else u = U2{u[0] >> bits | u[1] << (64 - bits), u[1] >> bits};
  return __builtin_bit_cast(typename Vec16<T>::type, u);
}
// The same in one step, with a branch.
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type load_vec(const T* row, int c, int n) {
  typedef typename Vec16<T>::type V;
  if (c + kVec<T> <= n) return *(const V*)(row + c);
  V v = {};
  if (c < n) {   // no lane where n is a multiple of the vector: the wave passes by
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
      if (c + j < n) v[j] = row[c + j];
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int c, int n, typename Vec16<T>::type v) {
  typedef typename Vec16<T>::type V;
  if (c + kVec<T> <= n) {
    *(V*)(row + c) = v;
    return;
  }
  if (c >= n) return;
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j)
    if (c + j < n) row[c + j] = v[j];
}

}  // namespace grpo
