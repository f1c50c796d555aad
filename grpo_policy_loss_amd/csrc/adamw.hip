// adamw.hip -- one AdamW step over many tensors in one launch.
//
// For every element, step t >= 1, g the gradient times an optional scale:
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   w = w - lr wd w - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
// w is the float32 master where there is one (the parameter is then its rounding), else the
// parameter.  The moments are float32, or 8-bit codes in blocks of 256 elements of one
// tensor with one float32 scale a = max |value| each:
//   m = sign(c) (c / 127)^2 a,  c = sign(m) floor(127 sqrt(|m| / a) + 1/2)
//   v = (c / 255)^4 a,          c = floor(255 (v / a)^(1/4) + 1/2), at least 1 where v > 0
// The powers spend the codes on the small values of a block: m spans 16129 : 1 and sqrt(v),
// which is what divides, 65025 : 1.  A positive v never reads back as 0, so the quotient
// never sees a zero under a live m (unless a is below float32's range).  A block with a value
// that is not finite has the scale NaN, so all of it reads back as NaN.
//
// With float32 moments the step is bound by memory: 20 to 30 bytes an element against some 20
// instructions (233M bf16 weights with masters: 1.09 to 1.21 ms from card to card, 5.8 to 6.4 TB/s).
// With 8-bit moments 10 bytes stand against some 80, a third of them in float64, and both count (67M
// bf16 weights: 175 to 181 us, 3.8 TB/s; 245 us with the definition of the codes worked out in every
// wave that has a root near a border).  One block takes a chunk of one tensor, 4 elements a lane and
// load, all loads of the chunk issued before its first use.
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "api.hpp"
#include "elem.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

// A block of 256 threads takes a chunk of STEPS * 1024 elements: 2048, or 4096 in plans of at least
// 2^26 elements with float32 moments.  2048 against 4096 elements, in us:
//   parameters, gradients        2^26 elements   2^27 elements
//   bf16, f32, masters           354   340       719   696   (8192: 723 against 689)
//   bf16, bf16, masters          296   299       675   656
//   bf16, f32                    238   231       567   548
//   bf16, bf16                   246   242       490   500
//   f32, f32                     318   309       645   631
//   f32, bf16                    272   271       603   596
// 2^24 with masters 83.3 and 83.5 us, 160 small tensors 10.1 and 11.2; moments in 8 bits are 5 %
// slower with 4096 at any size.
constexpr int kStep = 1024, kChunk = 2 * kStep, kLongChunk = 4 * kStep;
constexpr int64_t kMany = (int64_t)1 << 26;
constexpr int kQuantBlock = 256;    // elements per scale: one wave's load

// The image of a plan: this header, the tensors, then the first chunk of each tensor.
struct PlanHeader {
  uint64_t magic;
  int64_t count, chunks;
  int32_t param_dtype, grad_dtype, bits, master;
  int64_t chunk;               // elements
  int64_t o_tensors, o_first;
};
constexpr uint64_t kMagic = 0x314e414c50574441ull;

struct Hyper {
  double b1, b2, log_b1, log_b2;
  float lr, wd, eps;
  float step_size, inv_bc2;      // of the host's step and lr
  const int64_t* step_dev;       // non-null: the step is read here
  const float* lr_dev;
  const float* grad_scale;
};

template <typename T> struct Vec4;
template <> struct Vec4<float> {
  typedef __attribute__((ext_vector_type(4), aligned(4))) float type;
};
template <> struct Vec4<__bf16> {
  typedef __attribute__((ext_vector_type(4), aligned(2))) __bf16 type;
};
template <> struct Vec4<int8_t> {
  typedef __attribute__((ext_vector_type(4), aligned(1))) int8_t type;
};
template <> struct Vec4<uint8_t> {
  typedef __attribute__((ext_vector_type(4), aligned(1))) uint8_t type;
};

// Elements [e, e + 4) of n; those at n and behind it read as zero and are not written.  FULL:
// there are none.  Non-temporal, since a step passes once over what no cache holds until the
// next: 5 % off the 32-bit step and 10 % off the 8-bit one; 8-byte and smaller loads were
// faster with the caches' help (8-bit step 294 us against 279).
template <bool FULL, typename T>
__device__ __forceinline__ typename Vec4<T>::type load4(const T* p, int e, int n) {
  typedef const __attribute__((address_space(1))) typename Vec4<T>::type V;
  if (FULL || e + 4 <= n) {
    if constexpr (sizeof(T) == 4) return __builtin_nontemporal_load((V*)(p + e));
    else return *(V*)(p + e);
  }
  typename Vec4<T>::type v = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (e + j < n) v[j] = p[e + j];
  return v;
}
template <bool FULL, typename T>
__device__ __forceinline__ void store4(T* p, int e, int n, typename Vec4<T>::type v) {
  typedef __attribute__((address_space(1))) typename Vec4<T>::type V;
  if (FULL || e + 4 <= n) {
    __builtin_nontemporal_store(v, (V*)(p + e));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (e + j < n) p[e + j] = v[j];
}

// The wave's largest value, by row shifts and row broadcasts (no LDS).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define GRPO_STEP(ctrl, rows) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
  GRPO_STEP(0x111, 0xf);   // row_shr:1
  GRPO_STEP(0x112, 0xf);
  GRPO_STEP(0x114, 0xf);
  GRPO_STEP(0x118, 0xf);
  GRPO_STEP(0x142, 0xa);   // row_bcast:15
  GRPO_STEP(0x143, 0xc);   // row_bcast:31
#undef GRPO_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

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

// The codes from their definition, each operation rounded to float64 (none fused).
__device__ __forceinline__ float exact_m(double m, double a) {
#pragma clang fp contract(off)
  return fminf((float)floor(127.0 * sqrt(m / a) + 0.5), 127.f);
}
__device__ __forceinline__ float exact_v(double v, double a) {
#pragma clang fp contract(off)
  return fminf((float)floor(255.0 * sqrt(sqrt(v / a)) + 0.5), 255.f);
}

// The side of the nearer border b = c -+ 1/2 that the root r (of q, to 4 10^-5) is on, from
// q >= b^POWER in float64.  Within 10^-13 of it the definition's own roundings decide: `tie`.
template <int POWER>
__device__ __forceinline__ float side(float r, float c, double q, bool& tie) {
  const double b = (double)(r < c ? c - 0.5f : c + 0.5f);
  double t = b * b;
  if (POWER == 4) t *= t;
  tie |= fabs(q - t) <= 1e-13 * t;
  return (float)(q >= t ? b + 0.5 : b - 0.5);
}

// 1 / a to about 2^-52: the hardware's start and two Newton steps.
__device__ __forceinline__ double reciprocal(double a) {
  double r = __builtin_amdgcn_rcp(a);
  r = fma(r, fma(-a, r, 1.0), r);
  return fma(r, fma(-a, r, 1.0), r);
}

constexpr double kUnitM = 1.0 / 16129.0, kUnitV = 1.0 / 4228250625.0;   // 127^-2, 255^-4

// What a code stands for.  The last codes, 127 and 255, stand for a itself: their products with
// the constants round to 1.
__device__ __forceinline__ double value_m(int c, double a) {
  return (double)(c * abs(c)) * kUnitM * a;
}
__device__ __forceinline__ double value_v(unsigned c, double a) {
  const double s = (double)(c * c);
  return s * s * kUnitV * a;
}

// The moments after the step in float64, each product and sum rounded (none fused): a block's
// largest one is often a former a, and b1 a + (1 - b1) g then often lies just between two float32
// scales (one block in ten of those with b1 = 0.9), where the last bit of float64 decides.
__device__ __forceinline__ double next_m(double m, double x, double b1) {
#pragma clang fp contract(off)
  return m * b1 + x * (1.0 - b1);
}
__device__ __forceinline__ double next_v(double v, double x, double b2) {
#pragma clang fp contract(off)
  return v * b2 + x * x * (1.0 - b2);
}

// What is the same for every element.
struct Factors {
  float scale, decay, step_size, inv_bc2, eps;
  float b1, b2, a1, a2;
};

// m / (sqrt(v / (1 - b2^t)) + eps)
__device__ __forceinline__ float quotient(float m, float v, const Factors& f) {
  return m / (sqrtf(v * f.inv_bc2) + f.eps);
}

// The same with the hardware's root and reciprocal, good to a unit in the last place for normal
// numbers; a smaller root only matters beside an eps that is smaller still: `tiny`.
__device__ __forceinline__ float quick_quotient(float m, float v, const Factors& f, bool& tiny) {
  const float vh = v * f.inv_bc2;
  tiny |= !(vh >= 1.17549435e-38f);
  return m * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(vh) + f.eps);
}

template <typename P, typename G, int BITS, bool MASTER, int STEPS, bool FULL>
__device__ __forceinline__ void step_chunk(const grpo_adamw_tensor& t, int64_t base, const Hyper& h,
                                           const Factors& f) {
  const int n = FULL ? STEPS * kStep : (int)(t.n - base);
  P* param = (P*)t.param + base;
  const G* grad = (const G*)t.grad + base;
  float* master = t.master + (MASTER ? base : 0);
  typename Vec4<P>::type p[STEPS];
  typename Vec4<G>::type g[STEPS];
  typename Vec4<float>::type w[STEPS], m[STEPS], v[STEPS];
  typename Vec4<int8_t>::type mc[STEPS];
  typename Vec4<uint8_t>::type vc[STEPS];
  float ma[STEPS], va[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int e = (k * 256 + (int)threadIdx.x) * 4;
    g[k] = load4<FULL>(grad, e, n);
    if constexpr (MASTER) w[k] = load4<FULL>(master, e, n);
    else p[k] = load4<FULL>(param, e, n);
    if constexpr (BITS == 32) {
      m[k] = load4<FULL>((const float*)t.exp_avg + base, e, n);
      v[k] = load4<FULL>((const float*)t.exp_avg_sq + base, e, n);
    } else {
      mc[k] = load4<FULL>((const int8_t*)t.exp_avg + base, e, n);
      vc[k] = load4<FULL>((const uint8_t*)t.exp_avg_sq + base, e, n);
      const int64_t b = base / kQuantBlock + e / kQuantBlock;      // one scale per wave and step
      ma[k] = FULL || e < n ? t.exp_avg_scales[b] : 0.f;
      va[k] = FULL || e < n ? t.exp_avg_sq_scales[b] : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int e = (k * 256 + (int)threadIdx.x) * 4;
    float nm[4], nv[4];
    double dm[4], dv[4];
    if constexpr (BITS == 32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = (float)g[k][j] * f.scale;
        // fused by hand here and below: left to the compiler, which product is fused could differ
        // between whole and last chunks, and results then go by where a tensor ends
        nm[j] = fmaf(m[k][j], f.b1, x * f.a1);
        nv[j] = fmaf(v[k][j], f.b2, x * x * f.a2);
      }
    } else {
      // float64, so that the new codes are those of the exact moments
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double x = (double)(float)g[k][j] * (double)f.scale;
        dm[j] = next_m(value_m(mc[k][j], (double)ma[k]), x, h.b1);
        dv[j] = next_v(value_v(vc[k][j], (double)va[k]), x, h.b2);
        nm[j] = (float)dm[j];
        nv[j] = (float)dv[j];
      }
    }
    float u[4];
    bool tiny = BITS == 32;
    if constexpr (BITS == 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = quick_quotient(nm[j], nv[j], f, tiny);
    }
    if (tiny) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (BITS == 32 || !(nv[j] * f.inv_bc2 >= 1.17549435e-38f)) u[j] = quotient(nm[j], nv[j], f);
    }
    typename Vec4<P>::type np;
    typename Vec4<float>::type nw;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float old;
      if constexpr (MASTER) old = w[k][j];
      else old = (float)p[k][j];
      nw[j] = fmaf(-f.step_size, u[j], fmaf(-f.decay, old, old));
      np[j] = (P)nw[j];
    }
    store4<FULL>(param, e, n, np);
    if constexpr (MASTER) store4<FULL>(master, e, n, nw);
    if constexpr (BITS == 32) {
      store4<FULL>((float*)t.exp_avg + base, e, n, typename Vec4<float>::type{nm[0], nm[1], nm[2], nm[3]});
      store4<FULL>((float*)t.exp_avg_sq + base, e, n, typename Vec4<float>::type{nv[0], nv[1], nv[2], nv[3]});
    } else {
      // the block's largest magnitudes, as bits: above those of every finite value lie infinity
      // and NaN (lanes behind n hold zeros)
      uint32_t bits_m = 0, bits_v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bits_m = max(bits_m, __float_as_uint(nm[j]) & 0x7fffffffu);
        bits_v = max(bits_v, __float_as_uint(nv[j]) & 0x7fffffffu);
      }
      bits_m = wave_max(bits_m);
      bits_v = wave_max(bits_v);
      const bool bad_m = bits_m >= 0x7f800000u, bad_v = bits_v >= 0x7f800000u;
      if (bad_m)
        for (int j = 0; j < 4; ++j) dm[j] = nm[j] = 0.f;
      if (bad_v)
        for (int j = 0; j < 4; ++j) dv[j] = nv[j] = 0.f;
      const float top_m = __uint_as_float(bits_m), top_v = __uint_as_float(bits_v);
      const double to_m = bad_m || bits_m == 0 ? 0.0 : 16129.0 * reciprocal((double)top_m);
      const double to_v = bad_v || bits_v == 0 ? 0.0 : 4228250625.0 * reciprocal((double)top_v);
      float cm[4], cv[4], rm[4], rv[4], edge = 0.f;
      double qm[4], qv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        qm[j] = fabs(dm[j]) * to_m;
        qv[j] = dv[j] * to_v;
        rm[j] = __builtin_amdgcn_sqrtf((float)qm[j]);
        rv[j] = __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf((float)qv[j]));
        cm[j] = rintf(rm[j]);
        cv[j] = rintf(rv[j]);
        edge = fmaxf(edge, fmaxf(fabsf(rm[j] - cm[j]), fabsf(rv[j] - cv[j])));
      }
      // the roots are off by less than 4 10^-5 (two square roots of 1 ulp and the narrowing, up to
      // 255), so only those that near a border c + 1/2 need float64 (one step of a wave in twenty
      // has one), and only those on it the definition.  Exact halves are not rare: m / a is 1/4 where
      // the first step meets a gradient of a quarter of its block's largest.  A scale below the
      // normal numbers may be rounded so far that a root passes the last code.
      bool tie = bits_m - 1u < 0x7fffffu || bits_v - 1u < 0x7fffffu;   // a tiny scale, not 0
      if (edge > 0.49995f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cm[j] = side<2>(rm[j], cm[j], qm[j], tie);
          cv[j] = side<4>(rv[j], cv[j], qv[j], tie);
        }
      }
      if (tie) {
#pragma unroll 1   // one copy of the divisions: the kernel stays in the instruction cache
        for (int i = 0; i < 4; ++i) {
          double x = dm[0], y = dv[0];
#pragma unroll
          for (int j = 1; j < 4; ++j) x = i == j ? dm[j] : x, y = i == j ? dv[j] : y;
          const float em = exact_m(fabs(x), (double)top_m), ev = exact_v(y, (double)top_v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (i == j && bits_m != 0 && !bad_m) cm[j] = em;
            if (i == j && bits_v != 0 && !bad_v) cv[j] = ev;
          }
        }
      }
      typename Vec4<int8_t>::type om;
      typename Vec4<uint8_t>::type ov;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        om[j] = (int8_t)(int)__builtin_copysignf(cm[j], nm[j]);
        ov[j] = (uint8_t)max((unsigned)cv[j], qv[j] > 0.0 ? 1u : 0u);
      }
      store4<FULL>((int8_t*)t.exp_avg + base, e, n, om);
      store4<FULL>((uint8_t*)t.exp_avg_sq + base, e, n, ov);
      if ((threadIdx.x & 63) == 0 && (FULL || e < n)) {
        const int64_t b = base / kQuantBlock + e / kQuantBlock;
        t.exp_avg_scales[b] = bad_m ? __builtin_nanf("") : top_m;
        t.exp_avg_sq_scales[b] = bad_v ? __builtin_nanf("") : top_v;
      }
    }
  }
}

template <typename P, typename G, int BITS, bool MASTER, int STEPS>
__global__ void __launch_bounds__(256)
    k_adamw(const grpo_adamw_tensor* __restrict__ tensors, const int64_t* __restrict__ first,
            int count, Hyper h) {
  const int64_t chunk = blockIdx.x;
  const int at = owner_of(first, count, chunk);
  const grpo_adamw_tensor t = tensors[at];
  const int64_t base = (chunk - first[at]) * (STEPS * kStep);

  Factors f;
  float lr = h.lr;
  f.step_size = h.step_size;
  f.inv_bc2 = h.inv_bc2;
  f.eps = h.eps;
  if (h.lr_dev != nullptr) lr = *h.lr_dev;
  if (h.step_dev != nullptr) {
    // 1 - b^t = -expm1(t log b), the product in float64: 1 - b^t loses nothing near b = 1
    const int64_t s = *h.step_dev;
    const double td = (double)(s < 1 ? 1 : s);
    f.step_size = lr / -expm1f((float)(td * h.log_b1));
    f.inv_bc2 = 1.f / -expm1f((float)(td * h.log_b2));
  } else if (h.lr_dev != nullptr) {
    f.step_size = lr * h.step_size;            // the host passed 1 / (1 - b1^t)
  }
  f.scale = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  f.decay = lr * h.wd;
  f.b1 = (float)h.b1;
  f.b2 = (float)h.b2;
  f.a1 = (float)(1.0 - h.b1);
  f.a2 = (float)(1.0 - h.b2);
  if (base + STEPS * kStep <= t.n) step_chunk<P, G, BITS, MASTER, STEPS, true>(t, base, h, f);
  else step_chunk<P, G, BITS, MASTER, STEPS, false>(t, base, h, f);
}

// The float32 values of 8-bit moments: a block takes 2048 of them.
template <typename C>
__global__ void __launch_bounds__(256)
    k_moment_values(const C* __restrict__ codes, const float* __restrict__ scales, int64_t n,
                    float* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * kChunk;
  const int left = (int)min<int64_t>(kChunk, n - base);
  constexpr int STEPS = kChunk / kStep;
  typename Vec4<C>::type c[STEPS];
  float a[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int e = (k * 256 + (int)threadIdx.x) * 4;
    c[k] = load4<false>(codes + base, e, left);
    a[k] = e < left ? scales[base / kQuantBlock + e / kQuantBlock] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    typename Vec4<float>::type o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = (C)-1 < (C)0 ? (float)value_m((int)c[k][j], (double)a[k])
                          : (float)value_v((unsigned)c[k][j], (double)a[k]);
    store4<false>(out + base, (k * 256 + (int)threadIdx.x) * 4, left, o);
  }
}

template <typename P, typename G, bool MASTER>
void launch_adamw(const PlanHeader& hd, const char* plan, const Hyper& h, hipStream_t s) {
  const auto* tensors = (const grpo_adamw_tensor*)(plan + hd.o_tensors);
  const auto* first = (const int64_t*)(plan + hd.o_first);
  const auto kernel = hd.bits == 8                ? k_adamw<P, G, 8, MASTER, 2>
                      : hd.chunk == kLongChunk ? k_adamw<P, G, 32, MASTER, 4>
                                               : k_adamw<P, G, 32, MASTER, 2>;
  kernel<<<(unsigned)hd.chunks, 256, 0, s>>>(tensors, first, (int)hd.count, h);
}

size_t image_bytes(int64_t count) {
  return align_up(sizeof(PlanHeader)) + align_up((size_t)count * sizeof(grpo_adamw_tensor)) +
         align_up((size_t)count * sizeof(int64_t));
}

struct Range {
  uintptr_t from, to;
  bool written;
};

// Two ranges that share a byte, one of them written, would race.
bool any_overlap(std::vector<Range>& r) {
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

int fill_plan(const grpo_adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype,
              int bits, char* image) {
  const size_t ps = param_dtype == GRPO_F32 ? 4 : 2, gs = grad_dtype == GRPO_F32 ? 4 : 2;
  std::vector<Range> ranges;
  ranges.reserve((size_t)count * 7);
  PlanHeader hd{kMagic, count, 0, param_dtype, grad_dtype, bits, 0, kChunk, 0, 0};
  hd.o_tensors = (int64_t)align_up(sizeof(PlanHeader));
  hd.o_first = hd.o_tensors + (int64_t)align_up((size_t)count * sizeof(grpo_adamw_tensor));
  auto* first = (int64_t*)(image + hd.o_first);
  int64_t with = 0, without = 0, elements = 0;
  for (int64_t i = 0; i < count; ++i) {
    const grpo_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t)1 << 48)
      return fail(GRPO_ERR_INVALID_ARG, "tensor %lld has %lld elements", (long long)i,
                  (long long)t.n);
    if (t.n == 0) continue;
    const size_t n = (size_t)t.n, ss = (n + kQuantBlock - 1) / kQuantBlock * 4;
    const struct {
      const void* p;
      size_t bytes, align;
      bool written, needed;
      const char* name;
    } parts[] = {{t.param, n * ps, ps, true, true, "param"},
                 {t.grad, n * gs, gs, false, true, "grad"},
                 {t.master, n * 4, 4, true, false, "master"},
                 {t.exp_avg, n * (bits / 8), (size_t)bits / 8, true, true, "exp_avg"},
                 {t.exp_avg_sq, n * (bits / 8), (size_t)bits / 8, true, true, "exp_avg_sq"},
                 {t.exp_avg_scales, ss, 4, true, bits == 8, "exp_avg_scales"},
                 {t.exp_avg_sq_scales, ss, 4, true, bits == 8, "exp_avg_sq_scales"}};
    for (const auto& q : parts) {
      if (q.p == nullptr && q.needed)
        return fail(GRPO_ERR_INVALID_ARG, "null pointer: %s of tensor %lld", q.name, (long long)i);
      if (q.p == nullptr || (bits == 32 && &q >= &parts[5])) continue;
      const uintptr_t from = (uintptr_t)q.p;
      if (from % q.align != 0)
        return fail(GRPO_ERR_INVALID_ARG, "%s of tensor %lld is not aligned to its elements",
                    q.name, (long long)i);
      ranges.push_back({from, from + q.bytes, q.written});
    }
    (t.master != nullptr ? with : without) += 1;
    hd.chunks += (t.n + kChunk - 1) / kChunk;
    elements += t.n;
  }
  if (with != 0 && without != 0)
    return fail(GRPO_ERR_INVALID_ARG, "%lld tensors have a master and %lld have none: all or none",
                (long long)with, (long long)without);
  if (with != 0 && param_dtype == GRPO_F32)
    return fail(GRPO_ERR_INVALID_ARG, "a float32 parameter takes no master");
  if (hd.chunks > kMaxBlocks)
    return fail(GRPO_ERR_UNSUPPORTED, "more than 2^24 - 1 chunks of %d elements", kChunk);
  if (any_overlap(ranges))
    return fail(GRPO_ERR_INVALID_ARG, "two of the tensors overlap (the same one twice?)");
  hd.master = with != 0;
  if (bits == 32 && elements >= kMany) hd.chunk = kLongChunk;
  hd.chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    first[i] = hd.chunks;
    hd.chunks += (tensors[i].n + hd.chunk - 1) / hd.chunk;
  }
  memcpy(image, &hd, sizeof hd);
  if (count > 0) memcpy(image + hd.o_tensors, tensors, (size_t)count * sizeof(grpo_adamw_tensor));
  return GRPO_OK;
}

}  // namespace
}  // namespace grpo

using grpo::fail;

extern "C" {

size_t grpo_adamw_plan_bytes(int64_t count) {
  return count < 0 || count > grpo::kMaxTensors ? 0 : grpo::image_bytes(count);
}

int grpo_adamw_plan(const grpo_adamw_tensor* tensors, int64_t count, int param_dtype,
                    int grad_dtype, int state_bits, void* image, size_t image_bytes) {
  grpo::clear_error();
  if (count < 0 || count > grpo::kMaxTensors)
    return fail(GRPO_ERR_INVALID_ARG, "count %lld is not in [0, 2^24]", (long long)count);
  if (count > 0) GRPO_CHECK_PTR(tensors);
  GRPO_CHECK_PTR(image);
  for (int dt : {param_dtype, grad_dtype})
    if (dt != GRPO_F32 && dt != GRPO_BF16)
      return fail(GRPO_ERR_INVALID_ARG, "dtype %d is neither GRPO_F32 nor GRPO_BF16", dt);
  if (state_bits != 8 && state_bits != 32)
    return fail(GRPO_ERR_INVALID_ARG, "state_bits %d is neither 8 nor 32", state_bits);
  if (image_bytes < grpo::image_bytes(count))
    return fail(GRPO_ERR_WORKSPACE, "the plan's image needs %zu bytes, got %zu",
                grpo::image_bytes(count), image_bytes);
  try {
    return grpo::fill_plan(tensors, count, param_dtype, grad_dtype, state_bits, (char*)image);
  } catch (const std::bad_alloc&) {
    return fail(GRPO_ERR_WORKSPACE, "out of host memory");
  }
}

int grpo_adamw(const void* image, const void* plan, const grpo_adamw_opts* opts, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(image);
  GRPO_CHECK_PTR(opts);
  grpo::PlanHeader hd;
  memcpy(&hd, image, sizeof hd);
  if (hd.magic != grpo::kMagic)
    return fail(GRPO_ERR_INVALID_ARG, "image was not filled by grpo_adamw_plan");
  const grpo_adamw_opts& o = *opts;
  const double nonneg[] = {o.lr, o.eps, o.weight_decay};
  for (double x : nonneg)
    if (!(x >= 0.0 && x <= FLT_MAX))
      return fail(GRPO_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite in float32 and >= 0 "
                  "(%g, %g, %g)", o.lr, o.eps, o.weight_decay);
  if (!(o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0))
    return fail(GRPO_ERR_INVALID_ARG, "betas must be in [0, 1) (%g, %g)", o.beta1, o.beta2);
  if (o.step_dev == nullptr && o.step < 1)
    return fail(GRPO_ERR_INVALID_ARG, "step %lld: the first step is 1", (long long)o.step);
  if (hd.chunks == 0) return GRPO_OK;
  GRPO_CHECK_PTR(plan);
  if ((uintptr_t)plan % 8 != 0)
    return fail(GRPO_ERR_INVALID_ARG, "the plan's device copy is not 8-byte aligned");
  grpo::Hyper h{};
  h.b1 = o.beta1;
  h.b2 = o.beta2;
  h.log_b1 = log(o.beta1);
  h.log_b2 = log(o.beta2);
  h.lr = (float)o.lr;
  h.wd = (float)o.weight_decay;
  // a positive eps stays one: 0 / 0 is NaN.  (The root beside it is 0 or above 10^-23.)
  h.eps = o.eps > 0.0 ? fmaxf((float)o.eps, FLT_MIN) : 0.f;
  h.step_dev = o.step_dev;
  h.lr_dev = o.lr_dev;
  h.grad_scale = o.grad_scale;
  if (o.step_dev == nullptr) {
    const double bc1 = -expm1((double)o.step * h.log_b1), bc2 = -expm1((double)o.step * h.log_b2);
    h.step_size = (float)((o.lr_dev != nullptr ? 1.0 : o.lr) / bc1);
    h.inv_bc2 = (float)(1.0 / bc2);
  }
  hipStream_t s = (hipStream_t)stream;
  grpo::ScopedKernelTimer timer(grpo::KK_ADAMW, s);
  const char* p = (const char*)plan;
  if (hd.param_dtype == GRPO_F32) {
    if (hd.grad_dtype == GRPO_F32) grpo::launch_adamw<float, float, false>(hd, p, h, s);
    else grpo::launch_adamw<float, __bf16, false>(hd, p, h, s);
  } else if (hd.master) {
    if (hd.grad_dtype == GRPO_F32) grpo::launch_adamw<__bf16, float, true>(hd, p, h, s);
    else grpo::launch_adamw<__bf16, __bf16, true>(hd, p, h, s);
  } else {
    if (hd.grad_dtype == GRPO_F32) grpo::launch_adamw<__bf16, float, false>(hd, p, h, s);
    else grpo::launch_adamw<__bf16, __bf16, false>(hd, p, h, s);
  }
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

int grpo_moment_values(const void* codes, const float* scales, int64_t n, int squared, float* out,
                       void* stream) {
  grpo::clear_error();
  if (n < 0) return fail(GRPO_ERR_INVALID_ARG, "n must not be negative");
  if (squared != 0 && squared != 1)
    return fail(GRPO_ERR_INVALID_ARG, "squared must be 0 or 1");
  if (n == 0) return GRPO_OK;
  GRPO_CHECK_PTR(codes);
  GRPO_CHECK_PTR(scales);
  GRPO_CHECK_PTR(out);
  if (n > grpo::kMaxBlocks * grpo::kChunk) return fail(GRPO_ERR_UNSUPPORTED, "n is too large");
  const int64_t blocks = (n + grpo::kChunk - 1) / grpo::kChunk;
  hipStream_t s = (hipStream_t)stream;
  grpo::ScopedKernelTimer timer(grpo::KK_MOMENT_VALUES, s);
  if (squared)
    grpo::k_moment_values<uint8_t><<<(unsigned)blocks, 256, 0, s>>>((const uint8_t*)codes, scales,
                                                                    n, out);
  else
    grpo::k_moment_values<int8_t><<<(unsigned)blocks, 256, 0, s>>>((const int8_t*)codes, scales, n,
                                                                   out);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

}  // extern "C"
