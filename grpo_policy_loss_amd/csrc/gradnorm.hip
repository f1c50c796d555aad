// gradnorm.hip -- the norm of many gradients as one vector, the factor that clips it, and
// clipping in place.
//
//   norm = sqrt(sum g^2) or max |g|,  scale = min(1, max_norm / (norm + 1e-6))
// The optimizer's step takes the factor as its grad_scale, so a step that clips reads each
// gradient once more and writes none.  Bound by memory: 4 or 2 bytes an element against a
// conversion and a fused product in float64, in which no square overflows or underflows: 233M
// float32 in 140 us (6.7 TB/s), 68M bfloat16 in 29 (4.7) and clipped in 48 (5.6).
// Blocks take even shares of the chunks, one after the other, so that at most kBlocks partial
// results are left to a second launch of one block (none where one block took everything).
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "api.hpp"
#include "elem.hpp"
#include "plan.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

constexpr int kLanes = 256;       // threads of a chunk
constexpr int kChunk = 8192;      // elements: 8 loads of 16 bytes a thread in float32, 4 in bfloat16
constexpr int kClip = 2048;       // elements that a block clips: 332 us for 233M in float32, 340 and 357 of 4096 and 8192
constexpr int64_t kMaxChunks = kMaxBlocks / (kChunk / kClip);
constexpr int kBlocks = 2048;     // 8 on each of 256 CUs (4: 171 against 163 us for 233M in float32, 16: 162)
constexpr int kAlone = 1024;      // threads of the one block that needs no second launch
constexpr int kAloneChunks = 16;  // and the most chunks it takes

// The image of a plan: this header, the tensors, then the first chunk of each tensor.
struct GradHeader {
  uint64_t magic;
  int64_t count, chunks;
  int64_t o_tensors, o_first;
};
constexpr uint64_t kMagic = 0x314e414c50475247ull;

// A running sum of squares, or a running largest magnitude: the bits of one, above those of every
// finite value lie infinity and NaN.
template <int KIND> struct Running;
template <> struct Running<GRPO_GRAD_NORM_L2> {
  typedef double type;
  static __device__ __forceinline__ void add(type& r, float x) { r = fma((double)x, (double)x, r); }
  static __device__ __forceinline__ void join(type& r, type x) { r += x; }
  static __device__ __forceinline__ double norm(type r) { return sqrt(r); }
};
template <> struct Running<GRPO_GRAD_NORM_MAX> {
  typedef uint32_t type;
  static __device__ __forceinline__ void add(type& r, float x) { r = max(r, __float_as_uint(x) & 0x7fffffffu); }
  static __device__ __forceinline__ void join(type& r, type x) { r = max(r, x); }
  static __device__ __forceinline__ double norm(type r) { return (double)__uint_as_float(r); }
};

// A chunk of n elements (FULL: kChunk of them): all loads first.  Non-temporal, since whole gradients
// rarely stay in a cache until the optimizer reads them: 142 against 162 us for 233M in float32, 30
// against 33 for 68M in bfloat16 (and clipped after it 83 against 84).
template <int KIND, typename T, bool FULL>
__device__ __forceinline__ void add_chunk(const T* p, int n, typename Running<KIND>::type& r) {
  constexpr int kSteps = kChunk / (kLanes * kVec<T>);
  const int lane = threadIdx.x & (kLanes - 1);
  typename Vec16<T>::type v[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int e = (k * kLanes + lane) * kVec<T>;
    v[k] = FULL ? __builtin_nontemporal_load((const typename Vec16<T>::type*)(p + e)) : load_vec(p, e, n);
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) Running<KIND>::add(r, (float)v[k][j]);
}

template <int KIND>
__device__ __forceinline__ typename Running<KIND>::type block_join(typename Running<KIND>::type r) {
  __shared__ typename Running<KIND>::type waves[kAlone / 64];
  for (int o = 32; o >= 1; o >>= 1) Running<KIND>::join(r, __shfl_xor(r, o, 64));
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = r;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < (int)blockDim.x / 64; ++w) Running<KIND>::join(r, waves[w]);
  return r;
}

__device__ __forceinline__ void result(double n, double max_norm, float* norm, float* scale) {
  *norm = (float)n;
  const double s = max_norm / (n + 1e-6);
  *scale = max_norm == 0.0 || s >= 1.0 ? 1.f : (float)s;     // NaN stays
}

// kLanes threads take the chunks [share, share + 1) * chunks / shares.
template <int KIND, int THREADS>
__global__ void __launch_bounds__(THREADS)
    k_grad_norm(const grpo_grad_tensor* __restrict__ tensors, const int64_t* __restrict__ first,
                int count, int64_t chunks, double max_norm,
                typename Running<KIND>::type* __restrict__ parts, float* __restrict__ norm,
                float* __restrict__ scale) {
  constexpr int kPer = THREADS / kLanes;
  const int64_t shares = (int64_t)gridDim.x * kPer;
  const int64_t share = (int64_t)blockIdx.x * kPer + __builtin_amdgcn_readfirstlane((int)threadIdx.x / kLanes);
  const int64_t end = (share + 1) * chunks / shares;
  int64_t c = share * chunks / shares;
  typename Running<KIND>::type r = 0;
  if (c < end) {
    int at = owner_of(first, count, c);
    for (;;) {
      const grpo_grad_tensor t = tensors[at];
      const int64_t from = first[at], until = min(end, at + 1 < count ? first[at + 1] : chunks);
      for (; c < until; ++c) {
        const int64_t base = (c - from) * kChunk;
        const bool full = base + kChunk <= t.n;
        const int n = full ? kChunk : (int)(t.n - base);
        if (t.dtype == GRPO_F32) {
          const float* p = (const float*)t.grad + base;
          if (full) add_chunk<KIND, float, true>(p, n, r);
          else add_chunk<KIND, float, false>(p, n, r);
        } else {
          const __bf16* p = (const __bf16*)t.grad + base;
          if (full) add_chunk<KIND, __bf16, true>(p, n, r);
          else add_chunk<KIND, __bf16, false>(p, n, r);
        }
      }
      if (c >= end) break;
      ++at;            // a tensor of no elements has no chunks: the loop passes it by
    }
  }
  r = block_join<KIND>(r);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) result(Running<KIND>::norm(r), max_norm, norm, scale);
  else parts[blockIdx.x] = r;
}

template <int KIND>
__global__ void __launch_bounds__(kAlone)
    k_grad_finish(const typename Running<KIND>::type* __restrict__ parts, int count, double max_norm,
                  float* __restrict__ norm, float* __restrict__ scale) {
  typename Running<KIND>::type r = 0;
  for (int i = threadIdx.x; i < count; i += kAlone) Running<KIND>::join(r, parts[i]);
  r = block_join<KIND>(r);
  if (threadIdx.x == 0) result(Running<KIND>::norm(r), max_norm, norm, scale);
}

// A block's part of a chunk, or what there is of it.
template <typename T>
__device__ __forceinline__ void clip_chunk(T* p, int n, float s) {
  constexpr int kSteps = kClip / (kLanes * kVec<T>);
  typename Vec16<T>::type v[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) v[k] = load_vec((const T*)p, (k * kLanes + (int)threadIdx.x) * kVec<T>, n);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[k][j] = (T)((float)v[k][j] * s);
    store_vec(p, (k * kLanes + (int)threadIdx.x) * kVec<T>, n, v[k]);
  }
}

__global__ void __launch_bounds__(kLanes)
    k_grad_clip(const grpo_grad_tensor* __restrict__ tensors, const int64_t* __restrict__ first,
                int count, const float* __restrict__ scale) {
  const float s = *scale;
  if (s == 1.f) return;
  const int64_t c = blockIdx.x / (kChunk / kClip);
  const int at = owner_of(first, count, c);
  const grpo_grad_tensor t = tensors[at];
  const int64_t base = (c - first[at]) * kChunk + (blockIdx.x % (kChunk / kClip)) * kClip;
  const int n = (int)min<int64_t>(kClip, t.n - base);
  if (n <= 0) return;
  if (t.dtype == GRPO_F32) clip_chunk((float*)t.grad + base, n, s);
  else clip_chunk((__bf16*)t.grad + base, n, s);
}

size_t image_bytes(int64_t count) {
  return align_up(sizeof(GradHeader)) + align_up((size_t)count * sizeof(grpo_grad_tensor)) +
         align_up((size_t)count * sizeof(int64_t));
}

int fill_plan(const grpo_grad_tensor* tensors, int64_t count, char* image) {
  std::vector<Range> ranges;
  ranges.reserve((size_t)count);
  GradHeader hd{kMagic, count, 0, 0, 0};
  hd.o_tensors = (int64_t)align_up(sizeof(GradHeader));
  hd.o_first = hd.o_tensors + (int64_t)align_up((size_t)count * sizeof(grpo_grad_tensor));
  auto* first = (int64_t*)(image + hd.o_first);
  for (int64_t i = 0; i < count; ++i) {
    const grpo_grad_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t)1 << 48)
      return fail(GRPO_ERR_INVALID_ARG, "tensor %lld has %lld elements", (long long)i, (long long)t.n);
    if (t.dtype != GRPO_F32 && t.dtype != GRPO_BF16)
      return fail(GRPO_ERR_INVALID_ARG, "dtype %d of tensor %lld is neither GRPO_F32 nor GRPO_BF16", (int)t.dtype,
                  (long long)i);
    first[i] = hd.chunks;
    if (t.n == 0) continue;
    const size_t es = t.dtype == GRPO_F32 ? 4 : 2;
    if (t.grad == nullptr) return fail(GRPO_ERR_INVALID_ARG, "null pointer: tensor %lld", (long long)i);
    if ((uintptr_t)t.grad % es != 0)
      return fail(GRPO_ERR_INVALID_ARG, "tensor %lld is not aligned to its elements", (long long)i);
    ranges.push_back({(uintptr_t)t.grad, (uintptr_t)t.grad + (size_t)t.n * es, true});
    hd.chunks += (t.n + kChunk - 1) / kChunk;
    if (hd.chunks > kMaxChunks)
      return fail(GRPO_ERR_UNSUPPORTED, "more than 2^22 - 1 chunks of %d elements", kChunk);
  }
  if (any_overlap(ranges))
    return fail(GRPO_ERR_INVALID_ARG, "two of the tensors overlap (the same one twice?)");
  memcpy(image, &hd, sizeof hd);
  if (count > 0) memcpy(image + hd.o_tensors, tensors, (size_t)count * sizeof(grpo_grad_tensor));
  return GRPO_OK;
}

int read_plan(const void* image, const void* plan, GradHeader* hd) {
  GRPO_CHECK_PTR(image);
  memcpy(hd, image, sizeof *hd);
  if (hd->magic != kMagic) return fail(GRPO_ERR_INVALID_ARG, "image was not filled by grpo_grad_plan");
  if (hd->chunks == 0) return GRPO_OK;
  GRPO_CHECK_PTR(plan);
  if ((uintptr_t)plan % 8 != 0)
    return fail(GRPO_ERR_INVALID_ARG, "the plan's device copy is not 8-byte aligned");
  return GRPO_OK;
}

// Whether none of `of` shares a byte with a gradient of the plan.  A pass over the image on the host, 2 to 3 ns a
// tensor.
bool apart_from_gradients(const void* image, const GradHeader& hd, std::initializer_list<Memory> of) {
  const char* at = (const char*)image + hd.o_tensors;
  for (int64_t i = 0; i < hd.count; ++i) {
    grpo_grad_tensor t;
    memcpy(&t, at + i * (int64_t)sizeof t, sizeof t);
    const Memory g{t.n > 0 ? t.grad : nullptr, (size_t)t.n * (t.dtype == GRPO_F32 ? 4 : 2)};
    for (const Memory& m : of)
      if (share(g, m)) return false;
  }
  return true;
}

template <int KIND>
int grad_norm(const GradHeader& hd, const char* plan, double max_norm, float* norm, float* scale,
              void* ws, hipStream_t s) {
  typedef typename Running<KIND>::type R;
  const auto* tensors = (const grpo_grad_tensor*)(plan + hd.o_tensors);
  const auto* first = (const int64_t*)(plan + hd.o_first);
  const bool alone = hd.chunks <= kAloneChunks;
  const int blocks = alone ? 1 : (int)std::min<int64_t>(hd.chunks, kBlocks);
  {
    ScopedKernelTimer timer(KK_GRAD_NORM, s);
    if (alone)
      k_grad_norm<KIND, kAlone><<<1, kAlone, 0, s>>>(tensors, first, (int)hd.count, hd.chunks, max_norm, (R*)ws,
                                                    norm, scale);
    else
      k_grad_norm<KIND, kLanes><<<(unsigned)blocks, kLanes, 0, s>>>(tensors, first, (int)hd.count, hd.chunks,
                                                                   max_norm, (R*)ws, norm, scale);
    GRPO_HIP(hipGetLastError());
  }
  if (alone) return GRPO_OK;
  ScopedKernelTimer timer(KK_GRAD_FINISH, s);
  k_grad_finish<KIND><<<1, kAlone, 0, s>>>((const R*)ws, blocks, max_norm, norm, scale);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

}  // namespace
}  // namespace grpo

using grpo::fail;

extern "C" {

size_t grpo_grad_plan_bytes(int64_t count) {
  return count < 0 || count > grpo::kMaxTensors ? 0 : grpo::image_bytes(count);
}

int grpo_grad_plan(const grpo_grad_tensor* tensors, int64_t count, void* image,
                   size_t image_bytes) {
  grpo::clear_error();
  if (count < 0 || count > grpo::kMaxTensors)
    return fail(GRPO_ERR_INVALID_ARG, "count %lld is not in [0, 2^24]", (long long)count);
  if (count > 0) GRPO_CHECK_PTR(tensors);
  GRPO_CHECK_PTR(image);
  if (image_bytes < grpo::image_bytes(count))
    return fail(GRPO_ERR_WORKSPACE, "the plan's image needs %zu bytes, got %zu", grpo::image_bytes(count),
                image_bytes);
  try {
    return grpo::fill_plan(tensors, count, (char*)image);
  } catch (const std::bad_alloc&) {
    return fail(GRPO_ERR_WORKSPACE, "out of host memory");
  }
}

size_t grpo_grad_norm_workspace_bytes(void) { return grpo::kBlocks * sizeof(double); }

int grpo_grad_norm(const void* image, const void* plan, int kind, double max_norm, float* norm,
                   float* scale, void* workspace, size_t workspace_bytes, void* stream) {
  grpo::clear_error();
  grpo::GradHeader hd;
  const int st = grpo::read_plan(image, plan, &hd);
  if (st != GRPO_OK) return st;
  GRPO_CHECK_PTR(norm);
  GRPO_CHECK_PTR(scale);
  if (kind != GRPO_GRAD_NORM_L2 && kind != GRPO_GRAD_NORM_MAX)
    return fail(GRPO_ERR_INVALID_ARG, "kind %d is not 0 or 1", kind);
  if (!(max_norm >= 0.0 && max_norm <= FLT_MAX))
    return fail(GRPO_ERR_INVALID_ARG, "max_norm must be finite in float32 and >= 0 (%g)", max_norm);
  if (workspace == nullptr || workspace_bytes < grpo_grad_norm_workspace_bytes())
    return fail(GRPO_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", grpo_grad_norm_workspace_bytes(),
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  if ((uintptr_t)workspace % grpo::kAlign != 0)
    return fail(GRPO_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  const grpo::Memory n{norm, 4}, f{scale, 4}, ws{workspace, grpo_grad_norm_workspace_bytes()};
  if (!grpo::apart({n, f, ws}, {}) || !grpo::apart_from_gradients(image, hd, {n, f, ws}))
    return fail(GRPO_ERR_INVALID_ARG, "norm, scale or workspace overlaps a gradient or another of them");
  hipStream_t s = (hipStream_t)stream;
  const char* p = (const char*)plan;
  return kind == GRPO_GRAD_NORM_L2
             ? grpo::grad_norm<GRPO_GRAD_NORM_L2>(hd, p, max_norm, norm, scale, workspace, s)
             : grpo::grad_norm<GRPO_GRAD_NORM_MAX>(hd, p, max_norm, norm, scale, workspace, s);
}

int grpo_grad_clip(const void* image, const void* plan, const float* scale, void* stream) {
  grpo::clear_error();
  grpo::GradHeader hd;
  const int st = grpo::read_plan(image, plan, &hd);
  if (st != GRPO_OK) return st;
  GRPO_CHECK_PTR(scale);
  if (hd.chunks == 0) return GRPO_OK;
  if (!grpo::apart_from_gradients(image, hd, {{scale, 4}}))
    return fail(GRPO_ERR_INVALID_ARG, "scale is part of a gradient");
  hipStream_t s = (hipStream_t)stream;
  grpo::ScopedKernelTimer timer(grpo::KK_GRAD_CLIP, s);
  const char* p = (const char*)plan;
  const unsigned blocks = (unsigned)hd.chunks * (grpo::kChunk / grpo::kClip);
  grpo::k_grad_clip<<<blocks, grpo::kLanes, 0, s>>>(
      (const grpo_grad_tensor*)(p + hd.o_tensors), (const int64_t*)(p + hd.o_first), (int)hd.count, scale);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

}  // extern "C"
