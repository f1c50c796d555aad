// sample.hip -- one token per row of logits, from a given uniform number.
//
// A row x of V logits, z = x / T, weights e = exp(z - max z).  Tokens are ordered by (x down,
// index up); top-k keeps the first k, top-p of those the ones whose mass before them is less
// than p times the mass of those k, min-p of those the ones with e >= min_p.  The token is the
// lowest index whose running kept mass, in index order, exceeds u times the kept mass.  Its
// log-probability is that of the whole row: z - log sum exp z.
//
// A token is right or wrong, so what decides it is computed in 64 bits: a float32 sum over
// 150 000 tokens would move its borders past u in about one row of a hundred.  Where sums meet
// in any order (histograms), weights are whole multiples of 2^-42, whose sums over up to 2^20
// tokens are exact in 64 bits: no result depends on an order.
#include <math.h>

#include <algorithm>

#include "api.hpp"
#include "elem.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

constexpr int kSeg = 512;                  // tokens per segment: 8 a lane of one wave
constexpr int64_t kMaxVocab = 1 << 20;     // 2^20 weights of at most 2^42
constexpr int kMaxSegs = (int)(kMaxVocab / kSeg);
constexpr int kBins = 2048;

struct SampleArgs {
  const void* logits;
  const float* u;
  int64_t stride;
  int V, segs;
  double T, p, min_p;
  int k;
  const float* T_rows;
  const int32_t* k_rows;
  const float* p_rows;
  const float* min_p_rows;
  float* seg_max;      // [B, segs]
  double* seg_sum;     // [B, segs], relative to the segment's own maximum
  int32_t* token;
  float* lp;
};

// The parameters of one row, where 0 (or anything out of range in a device array) is off.
struct RowParams {
  double T, inv_T, p, min_p;
  int k;
  bool filtered;
};
__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t row) {
  RowParams r;
  r.T = a.T_rows != nullptr ? (double)a.T_rows[row] : a.T;
  if (r.T == 0.0) r.T = 1.0;
  r.inv_T = 1.0 / r.T;
  r.k = a.k_rows != nullptr ? a.k_rows[row] : a.k;
  if (r.k <= 0 || r.k >= a.V) r.k = 0;
  r.p = a.p_rows != nullptr ? (double)a.p_rows[row] : a.p;
  if (!(r.p > 0.0 && r.p < 1.0)) r.p = 0.0;
  r.min_p = a.min_p_rows != nullptr ? (double)a.min_p_rows[row] : a.min_p;
  if (!(r.min_p > 0.0)) r.min_p = 0.0;
  if (r.min_p > 1.0) r.min_p = 1.0;
  r.filtered = r.k != 0 || r.p != 0.0 || r.min_p != 0.0;
  return r;
}

// 8 consecutive logits from token c on; those at V and behind it read as -inf.  Minus zero
// becomes zero, its equal, so that the order of the bits is the order of the values.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int V, float (&x)[8]) {
  if (c + 8 <= V) {
#pragma unroll
    for (int i = 0; i < 8; i += kVec<T>) {
      const typename Vec16<T>::type v = load_vec(row, c + i, (int64_t)V);
#pragma unroll
      for (int j = 0; j < kVec<T>; ++j) x[i + j] = (float)v[j] + 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = c + j < V ? (float)row[c + j] + 0.f : -__builtin_huge_valf();
  }
}

template <typename V> __device__ __forceinline__ V wave_total(V v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_top(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
// Sums of the lanes below this one, and (total) of all.
template <typename V> __device__ __forceinline__ V wave_before(V v, V& total) {
  const int lane = threadIdx.x & 63;
  V up = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V t = __shfl_up(up, o, 64);
    if (lane >= o) up += t;
  }
  total = __shfl(up, 63, 64);
  return up - v;
}

// ---------------------------------------------------------------- maxima and sums
// One wave per segment of one row.  A NaN or +inf makes the segment's maximum NaN.
template <typename T>
__global__ void __launch_bounds__(256) k_sample_mass(SampleArgs a, int64_t waves) {
  const int lane = threadIdx.x & 63;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < waves; w += (int64_t)gridDim.x * 4) {
    const int64_t row = w / a.segs;
    const int seg = (int)(w - row * a.segs);
    float x[8];
    load8((const T*)a.logits + row * a.stride, seg * kSeg + lane * 8, a.V, x);
    float m = x[0];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m = fmaxf(m, x[j]);
      bad |= !(x[j] < __builtin_huge_valf());
    }
    m = wave_top(m);
    bad = __any(bad);
    double s = 0.0;
    if (!bad && m > -__builtin_huge_valf()) {
      const double inv_T = row_params(a, row).inv_T;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += exp(((double)x[j] - (double)m) * inv_T);
    }
    s = wave_total(s);
    if (lane == 0) {
      a.seg_max[w] = bad ? __builtin_nanf("") : m;
      a.seg_sum[w] = s;
    }
  }
}

// ---------------------------------------------------------------- the cut and the token
// A token's place in the order, larger first: the bits of x in ascending order, then the index
// reversed.
__device__ __forceinline__ uint64_t place(float x, int i) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t key = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((uint64_t)key << 20) | (uint32_t)(kMaxVocab - 1 - i);
}

// e in whole multiples of 2^-42: adding 2^10 puts its last bit at 2^-42 (rounded to nearest).
__device__ __forceinline__ uint64_t units(double e) {
  return (uint64_t)(__double_as_longlong(e + 1024.0) & ((1ll << 52) - 1));
}

struct RowState {
  float max;
  RowParams r;
  __device__ __forceinline__ double weight(float x) const {
    return exp(((double)x - (double)max) * r.inv_T);
  }
};

// Sums over the block's 1024 threads of the values before this thread's, and the total.
template <typename V>
__device__ __forceinline__ V block_before(V v, V* lds, V& total) {
  V wt;
  const V before = wave_before(v, wt);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = wt;
  __syncthreads();
  V off = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < (int)(threadIdx.x >> 6)) off += lds[i];
    total += lds[i];
  }
  return off + before;
}

struct Lds {
  uint64_t bins[kBins];
  double segs[kMaxSegs];
  uint64_t wave_u[16];
  double wave_d[16];
  uint64_t found_place, found_sum;
  int found;
};

// The place of the last kept token when tokens are kept in order while fewer than k were
// before (count), or while the mass before them is below `mass` units; only tokens at `floor`
// or above are looked at.  0 if all of them are kept.  Digit by digit over the 52 bits of a
// place: a histogram over the tokens that share the digits so far, and the bin that the border
// falls into.
template <typename T, bool MASS>
__device__ uint64_t find_cut(const T* x, int V, const RowState& st, uint64_t floor, uint64_t k,
                             double mass, Lds& l) {
  constexpr int width[5] = {11, 11, 10, 10, 10};
  uint64_t prefix = 0, above = 0;
  int shift = 52;
  for (int d = 0; d < 5; ++d) {
    const uint64_t top = prefix;             // digits so far
    const int upper = shift;
    shift -= width[d];
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += 1024) l.bins[i] = 0;
    __syncthreads();
    for (int c = threadIdx.x * 8; c < V; c += 1024 * 8) {
      float v[8];
      load8(x, c, V, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t pl = place(v[j], c + j);
        if (c + j >= V || pl < floor || (pl >> upper) != top) continue;
        const uint64_t add = MASS ? units(st.weight(v[j])) : 1;
        if (add) atomicAdd((unsigned long long*)&l.bins[(pl >> shift) & ((1 << width[d]) - 1)], (unsigned long long)add);
      }
    }
    __syncthreads();
    // from the top bin down: thread t holds bins n - 1 - 2t and n - 2 - 2t
    const int n = 1 << width[d], b0 = n - 1 - 2 * (int)threadIdx.x;
    const uint64_t s0 = b0 >= 0 ? l.bins[b0] : 0, s1 = b0 >= 1 ? l.bins[b0 - 1] : 0;
    uint64_t total;
    const uint64_t before = above + block_before<uint64_t>(s0 + s1, l.wave_u, total);
    if (threadIdx.x == 0) l.found = -1;
    __syncthreads();
    auto reaches = [&](uint64_t sum) { return MASS ? (double)sum >= mass : sum >= k; };
    if (s0 && !reaches(before) && reaches(before + s0)) {
      l.found = b0;
      l.found_sum = before;
    } else if (s1 && !reaches(before + s0) && reaches(before + s0 + s1)) {
      l.found = b0 - 1;
      l.found_sum = before + s0;
    }
    __syncthreads();
    if (l.found < 0) return 0;               // the border lies behind the last token
    above = l.found_sum;
    prefix = (top << width[d]) | (uint64_t)l.found;
  }
  return prefix;
}

// One block of 1024 threads per row.
template <typename T>
__global__ void __launch_bounds__(1024) k_sample_pick(SampleArgs a) {
  __shared__ Lds l;
  const int64_t row = blockIdx.x;
  const int V = a.V, lane = threadIdx.x & 63;
  const T* x = (const T*)a.logits + row * a.stride;
  const float* sm = a.seg_max + row * a.segs;
  const double* ss = a.seg_sum + row * a.segs;
  RowState st;
  st.r = row_params(a, row);

  // the row's maximum and mass: each thread takes two neighbouring segments
  float m[2];
  bool bad = false;
  float top = -__builtin_huge_valf();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * threadIdx.x + j;
    m[j] = i < a.segs ? sm[i] : -__builtin_huge_valf();
    bad |= m[j] != m[j];
    top = fmaxf(top, m[j]);
  }
  top = wave_top(top);
  bad = __any(bad);
  if (lane == 0) {
    l.wave_d[threadIdx.x >> 6] = (double)top;
    l.wave_u[threadIdx.x >> 6] = bad;
  }
  __syncthreads();
  bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, (float)l.wave_d[i]);
    bad |= l.wave_u[i] != 0;
  }
  st.max = top;
  if (bad || !(top > -__builtin_huge_valf()) || !(st.r.T > 0.0) || !(st.r.T < __builtin_huge_val())) {
    // nothing to draw from: a NaN or +inf, all -inf, or no temperature
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      a.lp[row] = __builtin_nanf("");
    }
    return;
  }
  double s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * threadIdx.x + j;
    s[j] = i < a.segs ? ss[i] * st.weight(m[j]) : 0.0;
  }
  double Z;
  block_before<double>(s[0] + s[1], l.wave_d, Z);

  const double u = fmin(fmax((double)a.u[row], 0.0), 1.0);
  uint64_t cut = 0;
  if (!st.r.filtered) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * threadIdx.x + j;
      l.segs[i] = s[j];
    }
    __syncthreads();
  } else {
    if (st.r.k != 0) cut = find_cut<T, false>(x, V, st, 0, (uint64_t)st.r.k, 0.0, l);
    if (st.r.p != 0.0) {
      // the mass of what top-k keeps, exactly
      uint64_t part = 0, zk;
      for (int c = threadIdx.x * 8; c < V; c += 1024 * 8) {
        float v[8];
        load8(x, c, V, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (place(v[j], c + j) >= cut && c + j < V) part += units(st.weight(v[j]));
      }
      block_before<uint64_t>(part, l.wave_u, zk);
      const uint64_t c2 = find_cut<T, true>(x, V, st, cut, 0, st.r.p * (double)zk, l);
      cut = c2 > cut ? c2 : cut;
    }
    // the kept mass of each segment, one wave a segment (whole multiples of 2^-42 below 2^62
    // of them in all: the doubles of a segment's at most 2^9 + 42 bits are exact)
    __syncthreads();
    for (int g = threadIdx.x >> 6; g < kMaxSegs; g += 16) {
      uint64_t part = 0;
      if (g < a.segs) {
        float v[8];
        const int c = g * kSeg + lane * 8;
        load8(x, c, V, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (c + j >= V || place(v[j], c + j) < cut) continue;
          const double e = st.weight(v[j]);
          if (e >= st.r.min_p) part += units(e);
        }
      }
      part = wave_total(part);
      if (lane == 0) l.segs[g] = (double)part * 0x1p-42;
    }
    __syncthreads();
  }
  const double s0 = l.segs[2 * threadIdx.x], s1 = l.segs[2 * threadIdx.x + 1];
  double sum;
  const double at = block_before<double>(s0 + s1, l.wave_d, sum);
  const double target = u * sum;
  // the lowest segment whose running mass exceeds the target, else the last that has any
  if (threadIdx.x == 0) l.found = kMaxSegs;
  __syncthreads();
  if (s0 > 0.0 && at + s0 > target) atomicMin(&l.found, 2 * (int)threadIdx.x);
  else if (s1 > 0.0 && at + s0 + s1 > target) atomicMin(&l.found, 2 * (int)threadIdx.x + 1);
  __syncthreads();
  int seg = l.found;
  if (seg == kMaxSegs) {
    __syncthreads();
    if (threadIdx.x == 0) l.found = 0;
    __syncthreads();
    if (s1 > 0.0) atomicMax(&l.found, 2 * (int)threadIdx.x + 1);
    else if (s0 > 0.0) atomicMax(&l.found, 2 * (int)threadIdx.x);
    __syncthreads();
    seg = l.found;
  }
  if ((int)threadIdx.x == seg / 2) l.wave_d[0] = seg & 1 ? at + s0 : at;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // its tokens, 8 a lane
  double rest = target - l.wave_d[0];
  float v[8];
  double e[8], mine = 0.0;
  const int c = seg * kSeg + lane * 8;
  load8(x, c, V, v);
  int last = -1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    e[j] = 0.0;
    if (c + j < V && place(v[j], c + j) >= cut) e[j] = st.weight(v[j]);
    if (st.r.filtered) e[j] = e[j] >= st.r.min_p ? (double)units(e[j]) * 0x1p-42 : 0.0;
    mine += e[j];
    if (e[j] > 0.0) last = j;
  }
  double wt;
  double run = wave_before(mine, wt);
  int hit = -1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    run += e[j];
    if (hit < 0 && e[j] > 0.0 && run > rest) hit = j;
  }
  uint64_t who = __ballot(hit >= 0);
  if (who == 0) {                       // the target is the mass itself (u = 1, a rounding)
    hit = last;
    who = __ballot(hit >= 0);
    who = who ? 1ull << (63 - __clzll(who)) : 1;
  }
  if (lane == __ffsll((unsigned long long)who) - 1) {
    const int j = hit < 0 ? 0 : hit;
    float z = v[0];
#pragma unroll
    for (int q = 1; q < 8; ++q)
      if (q == j) z = v[q];
    a.token[row] = c + j;
    a.lp[row] = (float)(((double)z - (double)st.max) * st.r.inv_T - log(Z));
  }
}

struct SamplePlan {
  int segs;
  size_t o_max, o_sum, total;
};
SamplePlan plan_sample(int64_t B, int64_t V) {
  SamplePlan p{};
  p.segs = (int)((V + kSeg - 1) / kSeg);
  p.o_max = 0;
  p.o_sum = align_up((size_t)(B * p.segs) * 4);
  p.total = p.o_sum + align_up((size_t)(B * p.segs) * 8);
  return p;
}

int check_sample(int64_t B, int64_t V, int64_t stride) {
  if (B <= 0 || V <= 0)
    return fail(GRPO_ERR_INVALID_ARG, "B and V must be positive (B=%lld V=%lld)", (long long)B,
                (long long)V);
  if (stride < V)
    return fail(GRPO_ERR_INVALID_ARG, "row_stride=%lld is below V=%lld", (long long)stride,
                (long long)V);
  if (V > kMaxVocab || B > (1 << 20))
    return fail(GRPO_ERR_UNSUPPORTED, "B and V may be at most 2^20");
  return GRPO_OK;
}

template <typename T>
hipError_t launch_sample(const SampleArgs& a, int64_t B, hipStream_t s) {
  const int64_t waves = B * a.segs;
  {
    ScopedKernelTimer t(KK_SAMPLE_MASS, s);
    const int64_t blocks = std::min<int64_t>((waves + 3) / 4, 1 << 20);
    k_sample_mass<T><<<(unsigned)blocks, 256, 0, s>>>(a, waves);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ScopedKernelTimer t(KK_SAMPLE_PICK, s);
  k_sample_pick<T><<<(unsigned)B, 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace grpo

using grpo::fail;

extern "C" {

size_t grpo_sample_workspace_bytes(int64_t B, int64_t V) {
  if (grpo::check_sample(B, V, V) != GRPO_OK) return 0;
  return grpo::plan_sample(B, V).total;
}

int grpo_sample(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                const float* u, const grpo_sample_opts* opts, int32_t* token, float* lp,
                void* workspace, size_t workspace_bytes, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(logits);
  GRPO_CHECK_PTR(u);
  GRPO_CHECK_PTR(token);
  GRPO_CHECK_PTR(lp);
  if (dtype != GRPO_F32 && dtype != GRPO_BF16)
    return fail(GRPO_ERR_INVALID_ARG, "dtype %d is neither GRPO_F32 nor GRPO_BF16", dtype);
  const int st = grpo::check_sample(B, V, row_stride);
  if (st != GRPO_OK) return st;
  const grpo_sample_opts none{};
  const grpo_sample_opts& o = opts == nullptr ? none : *opts;
  if (!isfinite(o.temperature) || o.temperature < 0.0)
    return fail(GRPO_ERR_INVALID_ARG, "temperature must be finite and >= 0, not %g", o.temperature);
  if (o.top_k < 0) return fail(GRPO_ERR_INVALID_ARG, "top_k must not be negative");
  if (!(o.top_p >= 0.0 && o.top_p <= 1.0 && o.min_p >= 0.0 && o.min_p <= 1.0))
    return fail(GRPO_ERR_INVALID_ARG, "top_p and min_p must be in [0, 1] (%g, %g)", o.top_p,
                o.min_p);
  const grpo::SamplePlan p = grpo::plan_sample(B, V);
  if (workspace == nullptr || workspace_bytes < p.total)
    return fail(GRPO_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", p.total,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  grpo::SampleArgs a{};
  a.logits = logits;
  a.u = u;
  a.stride = row_stride;
  a.V = (int)V;
  a.segs = p.segs;
  a.T = o.temperature;
  a.k = o.top_k;
  a.p = o.top_p;
  a.min_p = o.min_p;
  a.T_rows = o.temperature_rows;
  a.k_rows = o.top_k_rows;
  a.p_rows = o.top_p_rows;
  a.min_p_rows = o.min_p_rows;
  a.seg_max = (float*)((char*)workspace + p.o_max);
  a.seg_sum = (double*)((char*)workspace + p.o_sum);
  a.token = token;
  a.lp = lp;
  hipStream_t s = (hipStream_t)stream;
  GRPO_HIP(dtype == GRPO_BF16 ? grpo::launch_sample<__bf16>(a, B, s)
                              : grpo::launch_sample<float>(a, B, s));
  return GRPO_OK;
}

}  // extern "C"
