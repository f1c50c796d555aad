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
// in any order (histograms, lists), weights are whole multiples of 2^-42, whose sums over up to
// 2^20 tokens are exact in 64 bits: no result depends on an order.
//
// Rows by what their filters need, each with the fewest passes over the logits:
//   PLAIN    no filter: one pass for maxima and sums, then one segment of 2048 tokens.
//   LIST     top-k up to 2048 (or any filter on a row of at most 4096): the first pass keeps
//            the maximum of every 32 tokens; at least k of these are at or above the k-th
//            largest of them, so every kept token is, and only groups whose maximum is get
//            read again.  The candidates are sorted in LDS, where top-p and min-p are a cut.
//   MIN_P    the same with the bound max + T log min_p.
//   NUCLEUS  top-p alone: a histogram of the mass over 4096 bins of x finds the bin that the
//            cut falls into; one more pass sums what lies above and lists that bin's tokens.
//   GENERAL  everything else (larger k, lists that overflow as on rows of equal logits): the
//            cut digit by digit, one pass over the row for each of its 5 digits.
#include <math.h>

#include <algorithm>

#include "api.hpp"
#include "elem.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

constexpr int kCUs = 256;
constexpr int kSeg = 2048;                 // tokens per segment: one wave, 32 a lane
constexpr int64_t kMaxVocab = 1 << 20;     // 2^20 weights of at most 2^42
constexpr int kMaxSegs = (int)(kMaxVocab / kSeg);
constexpr int kBins = 2048;                // of one digit, and of the groups' maxima
constexpr int kNucleusBins = 4096;
constexpr int kList = 4096;                // candidates that are sorted in LDS
constexpr int kListK = 2048;               // largest top-k that goes by the groups' maxima

struct SampleArgs {
  const void* logits;
  const float* u;
  int64_t stride;
  int V, segs, splits;
  double T, p, min_p;
  int k;
  const float* T_rows;
  const int32_t* k_rows;
  const float* p_rows;
  const float* min_p_rows;
  float* seg_max;      // [B, segs]; NaN where the segment holds a NaN or +inf
  float* seg_min;      // [B, segs], of what is above -inf: NUCLEUS all tokens, LIST the groups' maxima
  double* seg_sum;     // [B, segs], relative to the segment's own maximum (not for NUCLEUS)
  float* grp_max;      // [B, segs, 64]: a lane's 32 tokens (LIST and MIN_P)
  // NUCLEUS
  uint64_t* hist;      // [B, splits, kNucleusBins]
  double* z_part;      // [B, splits]
  uint64_t* above;     // [B]: mass above the cut's bin
  uint64_t* whole;     // [B]: mass of the row
  uint64_t* seg_kept;  // [B, segs]: mass above the cut's bin, by segment
  int* listed;         // [B]: tokens in the cut's bin
  uint64_t* list;      // [B, kList]: their places
  int32_t* token;
  float* lp;
};

enum RowClass { PLAIN, LIST, MIN_P, NUCLEUS, GENERAL };

// The parameters of one row, where 0 (or anything out of range in a device array) is off.
struct RowParams {
  double T, rate, p, min_p;      // rate: log2(e) / T
  int k;
  RowClass cls;
};
__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t row) {
  RowParams r;
  r.T = a.T_rows != nullptr ? (double)a.T_rows[row] : a.T;
  if (r.T == 0.0) r.T = 1.0;
  r.rate = 1.4426950408889634 / r.T;
  r.k = a.k_rows != nullptr ? a.k_rows[row] : a.k;
  if (r.k <= 0 || r.k >= a.V) r.k = 0;
  r.p = a.p_rows != nullptr ? (double)a.p_rows[row] : a.p;
  if (!(r.p > 0.0 && r.p < 1.0)) r.p = 0.0;
  r.min_p = a.min_p_rows != nullptr ? (double)a.min_p_rows[row] : a.min_p;
  if (!(r.min_p > 0.0)) r.min_p = 0.0;
  if (r.min_p > 1.0) r.min_p = 1.0;
  if (r.k == 0 && r.p == 0.0 && r.min_p == 0.0) r.cls = PLAIN;
  else if (a.V <= kList || (r.k != 0 && r.k <= kListK)) r.cls = LIST;
  else if (r.k != 0) r.cls = GENERAL;
  else r.cls = r.p != 0.0 ? NUCLEUS : MIN_P;
  return r;
}

// 2^t for t <= 0: t = n + f with n whole and |f| <= 1/2, and 2^f by its interpolation at the
// Chebyshev points of degree 10 (relative error below 5e-16).  Below 2^-1000 it stays at
// 2^-1000: nothing beside the row's maximum, whose weight is 1.
__device__ __forceinline__ double pow2_down(double t) {
  t = fmax(t, -1000.0);
  const double magic = 0x1.8p52, shifted = t + magic;
  const double f = t - (shifted - magic);
  double q = 0x1.e6063f7217bc6p-28;
  q = fma(q, f, 0x1.b675bca4eeebbp-24);
  q = fma(q, f, 0x1.62bfd47773353p-20);
  q = fma(q, f, 0x1.ffcb54062e698p-17);
  q = fma(q, f, 0x1.430913096fd9fp-13);
  q = fma(q, f, 0x1.5d87fe9d7a584p-10);
  q = fma(q, f, 0x1.3b2ab6fba1ddap-7);
  q = fma(q, f, 0x1.c6b08d703ce49p-5);
  q = fma(q, f, 0x1.ebfbdff82c598p-3);
  q = fma(q, f, 0x1.62e42fefa3a19p-1);
  q = fma(q, f, 1.0);
  // n into the exponent: q is in [0.7, 1.5] and n at least -1000
  const int n = (int)(uint32_t)__double_as_longlong(shifted);
  return __hiloint2double(__double2hiint(q) + n * (1 << 20), __double2loint(q));
}

// 8 consecutive logits from token c on; those at V and behind it read as -inf.  Loading and
// unpacking are apart, so that loads can be under way while others are worked on.
template <typename T> struct Raw8 {
  typename Vec16<T>::type v[8 / kVec<T>];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* row, int c, int V) {
  Raw8<T> r;
  if (c + 8 <= V) {
#pragma unroll
    for (int i = 0; i < 8; i += kVec<T>) r.v[i / kVec<T>] = *(const typename Vec16<T>::type*)(row + c + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const T v = row[min(c + j, V - 1)];
      r.v[j / kVec<T>][j % kVec<T>] = c + j < V ? v : (T)-__builtin_huge_valf();
    }
  }
  return r;
}
// Minus zero becomes zero, its equal: the order of the bits is then the order of the values.
template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (float)r.v[j / kVec<T>][j % kVec<T>] + 0.f;
}
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int V, float (&x)[8]) {
  unpack(load8(row, c, V), x);
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
__device__ __forceinline__ float wave_low(float v) { return -wave_top(-v); }
// Of values that ascend with the lane: the least `hit` (INT32_MAX: none) and the largest `last`
// (-1: none) of the wave, in every lane.  (An LDS atomic on one address would run lane by lane.)
__device__ __forceinline__ void first_and_last(int& hit, int& last) {
  const uint64_t h = __ballot(hit != INT32_MAX), t = __ballot(last >= 0);
  hit = h ? __shfl(hit, __ffsll((unsigned long long)h) - 1, 64) : INT32_MAX;
  last = t ? __shfl(last, 63 - __clzll((unsigned long long)t), 64) : -1;
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
// One wave per segment of one row; the next segment's loads are under way while this one's
// weights are summed.  About 20 float64 instructions a token are as many as the loads leave
// time for.
template <typename T> struct RawSeg {
  Raw8<T> q[4];
};
template <typename T>
__device__ __forceinline__ RawSeg<T> load_seg(const SampleArgs& a, int64_t row, int seg) {
  const int c = seg * kSeg + (threadIdx.x & 63) * 8;
  RawSeg<T> r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r.q[q] = load8((const T*)a.logits + row * a.stride, c + q * 512, a.V);
  return r;
}

template <typename T>
__global__ void __launch_bounds__(256) k_sample_mass(SampleArgs a, int64_t waves) {
  const int lane = threadIdx.x & 63;
  int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= waves) return;
  const int64_t step = (int64_t)gridDim.x * 4;
  RawSeg<T> next = load_seg<T>(a, w / a.segs, (int)(w % a.segs));
  for (;;) {
    float x[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q) unpack(next.q[q], x[q]);
    const bool more = w + step < waves;
    if (more) next = load_seg<T>(a, (w + step) / a.segs, (int)((w + step) % a.segs));
    const RowParams r = row_params(a, w / a.segs);
    float m = x[0][0], low;
    bool nan = false;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m = fmaxf(m, x[q][j]);
        nan |= x[q][j] != x[q][j];
      }
    low = m > -__builtin_huge_valf() ? m : __builtin_huge_valf();
    if (r.cls == LIST || r.cls == MIN_P) a.grp_max[w * 64 + lane] = m;
    if (r.cls == NUCLEUS) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[q][j] > -__builtin_huge_valf()) low = fminf(low, x[q][j]);
    }
    if (r.cls != PLAIN) low = wave_low(low);
    m = wave_top(m);
    const bool bad = __any(nan) || m == __builtin_huge_valf();
    double s = 0.0;
    if (r.cls != NUCLEUS && m > -__builtin_huge_valf()) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += pow2_down(((double)x[q][j] - (double)m) * r.rate);
      s = wave_total(s);
    }
    if (lane == 0) {
      a.seg_max[w] = bad ? __builtin_nanf("") : m;
      a.seg_min[w] = low;
      a.seg_sum[w] = s;
    }
    if (!more) return;
    w += step;
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

__device__ __forceinline__ float value_at(uint64_t place) {
  const uint32_t key = (uint32_t)(place >> 20);
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int index_at(uint64_t place) {
  return (int)(kMaxVocab - 1) - (int)(place & (kMaxVocab - 1));
}

struct RowState {
  float max;
  RowParams r;
  __device__ __forceinline__ double weight(float x) const {
    return pow2_down(((double)x - (double)max) * r.rate);
  }
};

// Bins of x from the maximum down, in float32: rounding keeps the order, so the bins are in the
// order of x.  -inf and what lies below the last bin's lower end are in the last bin.
struct Binning {
  float max, scale;
  int last;
  __device__ __forceinline__ Binning(float top, float range, int bins) : max(top), last(bins - 1) {
    scale = (float)last / range;
    if (!(scale < __builtin_huge_valf())) scale = 0.f;
  }
  __device__ __forceinline__ int operator()(float x) const {
    return (int)fminf((max - x) * scale, (float)last);   // fminf drops the NaN of inf * 0
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

// A row's maximum over its segments, whether it holds a NaN or +inf, and its minimum above
// -inf, for a block of 1024 threads (lds: 16 of each).
struct RowRange {
  float top, low;
  bool bad;
};
__device__ __forceinline__ RowRange row_range(const SampleArgs& a, int64_t row, float (*lds)[16]) {
  const int i = threadIdx.x;
  RowRange r;
  r.top = i < a.segs ? a.seg_max[row * a.segs + i] : -__builtin_huge_valf();
  r.low = i < a.segs ? a.seg_min[row * a.segs + i] : __builtin_huge_valf();
  r.bad = __any(r.top != r.top);
  r.top = wave_top(r.top);
  r.low = wave_low(r.low);
  if ((threadIdx.x & 63) == 0) {
    lds[0][i >> 6] = r.top;
    lds[1][i >> 6] = r.low;
    lds[2][i >> 6] = r.bad ? 1.f : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    r.top = fmaxf(r.top, lds[0][w]);
    r.low = fminf(r.low, lds[1][w]);
    r.bad |= lds[2][w] != 0.f;
  }
  return r;
}
// Whether there is anything to draw from.
__device__ __forceinline__ bool drawable(const RowRange& g, const RowParams& r) {
  return !g.bad && g.top > -__builtin_huge_valf() && r.T > 0.0 && r.T < __builtin_huge_val();
}
// Over 30 T below the maximum, 2^20 tokens weigh less than 10^-6 of it.
__device__ __forceinline__ Binning nucleus_bins(const RowRange& g, const RowParams& r) {
  return Binning(g.top, fminf(g.top - g.low, (float)(30.0 * r.T)), kNucleusBins);
}

// ---------------------------------------------------------------- NUCLEUS
// Block (split, row): the mass of the split's tokens by bin.
template <typename T>
__global__ void __launch_bounds__(1024) k_sample_hist(SampleArgs a) {
  const int64_t row = blockIdx.y;
  RowState st;
  st.r = row_params(a, row);
  if (st.r.cls != NUCLEUS) return;
  __shared__ uint64_t bins[kNucleusBins];
  __shared__ float range[3][16];
  __shared__ double zs[16];
  const int per = (a.segs + a.splits - 1) / a.splits * kSeg;
  const int from = blockIdx.x * per, to = min(a.V, from + per);
  const T* x = (const T*)a.logits + row * a.stride;
  Raw8<T> next = {};
  if (from + (int)threadIdx.x * 8 < to) next = load8(x, from + threadIdx.x * 8, a.V);
  for (int i = threadIdx.x; i < kNucleusBins; i += 1024) bins[i] = 0;
  const RowRange g = row_range(a, row, range);      // its barrier is also the bins'
  if (!drawable(g, st.r)) return;
  st.max = g.top;
  const Binning bin = nucleus_bins(g, st.r);
  double z = 0.0;
  for (int c = from + threadIdx.x * 8; c < to; c += 1024 * 8) {
    float v[8];
    unpack(next, v);
    if (c + 1024 * 8 < to) next = load8(x, c + 1024 * 8, a.V);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double e = st.weight(v[j]);
      z += e;
      const uint64_t n = units(e);
      if (n) atomicAdd((unsigned long long*)&bins[bin(v[j])], (unsigned long long)n);
    }
  }
  double total;
  block_before<double>(z, zs, total);
  uint64_t* out = a.hist + (row * a.splits + blockIdx.x) * kNucleusBins;
  for (int i = threadIdx.x; i < kNucleusBins; i += 1024) out[i] = bins[i];
  if (threadIdx.x == 0) {
    a.z_part[row * a.splits + blockIdx.x] = total;
    if (blockIdx.x == 0) a.listed[row] = 0;
  }
}

// Block (split, row): the bin that the cut falls into, the mass above it by segment and the
// places of its tokens.
template <typename T>
__global__ void __launch_bounds__(1024) k_sample_gather(SampleArgs a) {
  const int64_t row = blockIdx.y;
  RowState st;
  st.r = row_params(a, row);
  if (st.r.cls != NUCLEUS) return;
  __shared__ float range[3][16];
  __shared__ uint64_t sums[16];
  __shared__ uint64_t mine[kList];
  __shared__ int found, count, at;
  const RowRange g = row_range(a, row, range);
  if (!drawable(g, st.r)) return;
  st.max = g.top;
  const Binning bin = nucleus_bins(g, st.r);
  // thread t holds bins 4t .. 4t + 3
  uint64_t h[4] = {0, 0, 0, 0}, total;
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) {
    const uint64_t* in = a.hist + (row * a.splits + s) * kNucleusBins + 4 * threadIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] += in[j];
  }
  if (threadIdx.x == 0) {
    found = kNucleusBins - 1;
    count = 0;
  }
  uint64_t run = block_before<uint64_t>(h[0] + h[1] + h[2] + h[3], sums, total);
  const double mass = st.r.p * (double)total;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (h[j] && (double)run < mass && (double)(run + h[j]) >= mass) {
      found = 4 * threadIdx.x + j;       // one thread's: the sums ascend
      if (blockIdx.x == 0) {
        a.above[row] = run;
        a.whole[row] = total;
      }
    }
    run += h[j];
  }
  __syncthreads();
  const int cut_bin = found, lane = threadIdx.x & 63;
  const int per = (a.segs + a.splits - 1) / a.splits;
  const int end = min(a.segs, (int)(blockIdx.x + 1) * per);
  for (int seg = blockIdx.x * per + (threadIdx.x >> 6); seg < end; seg += 16) {
    uint64_t part = 0;
    const RawSeg<T> raw = load_seg<T>(a, row, seg);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = seg * kSeg + q * 512 + lane * 8;
      float v[8];
      unpack(raw.q[q], v);
      unsigned in_cut = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int b = bin(v[j]);
        in_cut |= b == cut_bin && c + j < a.V ? 1u << j : 0u;
        if (b < cut_bin) {
          const double e = st.weight(v[j]);
          if (e >= st.r.min_p) part += units(e);
        }
      }
      if (__any(in_cut)) {
        int all = 0, slot = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t who = __ballot((in_cut >> j) & 1);
          slot += __popcll(who & ((1ull << lane) - 1));
          all += __popcll(who);
        }
        int first = 0;
        if (lane == 0) first = atomicAdd(&count, all);
        slot += __builtin_amdgcn_readfirstlane(first);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((in_cut >> j) & 1) {
            if (slot < kList) mine[slot] = place(v[j], c + j);
            ++slot;
          }
      }
    }
    part = wave_total(part);
    if (lane == 0) a.seg_kept[row * a.segs + seg] = part;
  }
  __syncthreads();
  const int n = count;
  if (threadIdx.x == 0) at = n ? atomicAdd(&a.listed[row], n) : 0;
  __syncthreads();
  // more than kList in all, or in this block: the pick sees the count and goes by digits
  for (int i = threadIdx.x; i < min(n, kList); i += 1024)
    if (at + i < kList) a.list[row * kList + at + i] = mine[i];
}

// ---------------------------------------------------------------- the pick
struct Lds {
  union {
    uint64_t bins[kBins];
    uint64_t list[kList];
    unsigned counts[kBins];
  };
  union {
    uint64_t segs_u[kMaxSegs];
    double segs[kMaxSegs];
  };
  uint64_t wave_u[16];
  double wave_d[16];
  float range[3][16];
  uint64_t found_sum;
  int found, count;
  int first[16], last[16];
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

// Sorts list[0, n) downwards; places differ.  Up to 512: each thread counts the larger ones.
// Above: bitonic, filled with 0 up to a power of two.
__device__ __forceinline__ void sort_list(uint64_t* list, int n) {
  __syncthreads();
  if (n <= 512) {
    const int t = threadIdx.x;
    uint64_t own = 0;
    int rank = 0;
    if (t < n) {
      own = list[t];
#pragma unroll 8
      for (int i = 0; i < n; ++i) rank += list[i] > own;
    }
    __syncthreads();
    if (t < n) list[rank] = own;
    __syncthreads();
    return;
  }
  int size = 1024;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += 1024) list[i] = 0;
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
#pragma unroll 1
      for (int t = threadIdx.x; t < size / 2; t += 1024) {
        const int lo = ((t & ~(j - 1)) << 1) | (t & (j - 1)), hi = lo | j;
        const uint64_t p = list[lo], q = list[hi];
        if ((p < q) == ((lo & k) == 0)) {
          list[lo] = q;
          list[hi] = p;
        }
      }
    }
  __syncthreads();
}

// The tokens that may be kept, into l.list; their number (over kList: too many).  A group is
// 32 tokens that one lane of k_sample_mass read; only groups whose maximum may be kept are
// read again.  `low`: the least of the groups' maxima.
template <typename T>
__device__ __forceinline__ int candidates(const SampleArgs& a, int64_t row, const T* x,
                                          const RowState& st, float low, Lds& l) {
  const int groups = a.segs * 64, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* gm = a.grp_max + row * groups;
  const float none = -__builtin_huge_valf();
  // 8192 groups at a time, thread t of wave w holding groups 1024 i + 64 w + lane (a segment's)
  float g[8];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = base + i * 1024 + (int)threadIdx.x;
      g[i] = at < groups ? gm[at] : none;
    }
  };
  load(0);
  Binning bin(st.max, 0.f, kBins);          // all that is above -inf into bin 0
  int last = kBins - 1;
  if (threadIdx.x == 0) {
    l.count = 0;
    l.found = -1;
  }
  if (st.r.cls == LIST && a.V > kList) {
    // bins over the range of the groups' maxima; the last one that the k largest reach into
    const Binning fine(st.max, st.max - low, kBins);
    l.counts[threadIdx.x] = l.counts[threadIdx.x + 1024] = 0;
    __syncthreads();
#pragma unroll 1
    for (int base = 0; base < groups; base += 8192) {
      if (base) load(base);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (g[i] > none) atomicAdd(&l.counts[fine(g[i])], 1u);
    }
    __syncthreads();
    const int b = 2 * threadIdx.x;
    const uint64_t c0 = l.counts[b], c1 = l.counts[b + 1], k = (uint64_t)st.r.k;
    uint64_t total;
    const uint64_t before = block_before<uint64_t>(c0 + c1, l.wave_u, total);
    if (before < k && before + c0 >= k) l.found = b;
    else if (before + c0 < k && before + c0 + c1 >= k) l.found = b + 1;
    __syncthreads();
    if (l.found >= 0) {                     // otherwise fewer groups than k: all of them
      last = l.found;
      bin = fine;
    }
    if (groups > 8192) load(0);
  } else {
    __syncthreads();
  }
  const bool by_weight = st.r.cls == MIN_P;
  auto wanted = [&](float v) {
    if (!(v > none)) return false;
    return by_weight ? st.weight(v) >= st.r.min_p : bin(v) <= last;
  };
#pragma unroll 1
  for (int base = 0; base < groups; base += 8192) {
    if (base) load(base);
    // a bit for each of this lane's groups that is wanted
    unsigned want = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) want |= wanted(g[i]) ? 1u << i : 0u;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      // of a segment's 64 groups the wanted ones, two at a time, 32 lanes each
      const int seg = (base + i * 1024) / 64 + wave;
      uint64_t todo = __ballot((want >> i) & 1u);
      while (todo) {
        const int one = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        const int two = todo ? __ffsll((unsigned long long)todo) - 1 : -1;
        todo &= todo - 1;
        const int gl = lane < 32 ? one : two;
        // tokens q * 512 + gl * 8 + j of the segment, q < 4 and j < 8
        const int k = lane & 31, c = seg * kSeg + (k >> 3) * 512 + gl * 8 + (k & 7);
        const bool in = gl >= 0 && c < a.V;
        const float v = in ? (float)x[c] + 0.f : none;
        const bool take = in && wanted(v);
        const uint64_t who = __ballot(take);
        int at = 0;
        if (lane == 0) at = atomicAdd(&l.count, __popcll(who));
        at = __builtin_amdgcn_readfirstlane(at) + __popcll(who & ((1ull << lane) - 1));
        if (take && at < kList) l.list[at] = place(v, c);
      }
    }
  }
  __syncthreads();
  return l.count;
}

// The place of the last kept token (0: all), from a row's sorted list of n places that follow
// on `above` units of mass; `whole` the mass that top-p is a share of (0: that of the list's
// first k).  Adds the kept tokens' masses to l.segs_u.
__device__ __forceinline__ uint64_t cut_list(const RowState& st, int n, uint64_t above, uint64_t whole, Lds& l) {
  sort_list(l.list, n);
  uint64_t m[4], sum = 0, total;
  double e[4];
  const int first = 4 * threadIdx.x, k = st.r.k != 0 ? min(n, st.r.k) : n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e[j] = first + j < k ? st.weight(value_at(l.list[first + j])) : 0.0;
    m[j] = first + j < k ? units(e[j]) : 0;
    sum += m[j];
  }
  if (threadIdx.x == 0) l.found = k - 1;
  uint64_t run = above + block_before<uint64_t>(sum, l.wave_u, total);
  if (st.r.p != 0.0) {
    const double mass = st.r.p * (double)(whole != 0 ? whole : total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // the token with which the mass reaches its share is the last kept one
      if (m[j] && (double)run < mass && (double)(run + m[j]) >= mass) l.found = first + j;
      run += m[j];
    }
  }
  __syncthreads();
  const int last = l.found;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (first + j <= last && m[j] && e[j] >= st.r.min_p)
      atomicAdd((unsigned long long*)&l.segs_u[index_at(l.list[first + j]) / kSeg], (unsigned long long)m[j]);
  const uint64_t cut = l.list[last];
  __syncthreads();
  return cut;
}

// Rows without filters, in a kernel of its own: one block of 256 threads per row, whose time is
// that of its four dependent loads.
template <typename T>
__global__ void __launch_bounds__(256) k_sample_plain(SampleArgs a) {
  __shared__ float tops[4];
  __shared__ int bad[4];
  __shared__ double mass[2][4];
  __shared__ int found[2][2][4];
  const int64_t row = blockIdx.x;
  const int V = a.V, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* x = (const T*)a.logits + row * a.stride;
  // thread t holds segments 2t and 2t + 1
  float m[2];
  double s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * threadIdx.x + j;
    m[j] = i < a.segs ? a.seg_max[row * a.segs + i] : -__builtin_huge_valf();
    s[j] = i < a.segs ? a.seg_sum[row * a.segs + i] : 0.0;
  }
  const double u = fmin(fmax((double)a.u[row], 0.0), 1.0);
  RowState st;
  st.r = row_params(a, row);
  RowRange g;
  g.bad = __any(m[0] != m[0] || m[1] != m[1]);
  g.top = wave_top(fmaxf(m[0], m[1]));
  if (lane == 0) {
    tops[wave] = g.top;
    bad[wave] = g.bad;
  }
  __syncthreads();
  g.top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  g.bad = bad[0] | bad[1] | bad[2] | bad[3];
  st.max = g.top;
  if (!drawable(g, st.r)) {
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      a.lp[row] = __builtin_nanf("");
    }
    return;
  }
  // where the running mass first exceeds u Z: the segment, then its token
  double Z = 0.0, target = 0.0;
  int seg = 0;
  float v[8];
  double e[8];
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int c = pass ? seg * kSeg + (int)threadIdx.x * 8 : 2 * (int)threadIdx.x;
    double own = 0.0;
    if (pass) {
      load8(x, c, V, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = v[j] > -__builtin_huge_valf() ? st.weight(v[j]) : 0.0;
        own += e[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        e[j] = s[j] > 0.0 ? s[j] * st.weight(m[j]) : 0.0;
        own += e[j];
      }
    }
    double wt, sum = 0.0;
    double run = wave_before(own, wt);
    if (lane == 63) mass[pass][wave] = wt;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < wave) run += mass[pass][i];
      sum += mass[pass][i];
    }
    if (!pass) {
      Z = sum;
      target = u * Z;
    }
    const double first = run;
    int hit = INT32_MAX, last = -1;
#pragma unroll
    for (int j = 0; j < (pass ? 8 : 2); ++j) {
      run += e[j];
      if (e[j] > 0.0) {
        if (run > target) hit = min(hit, c + j);
        last = c + j;
      }
    }
    first_and_last(hit, last);
    if (lane == 0) {
      found[pass][0][wave] = hit;
      found[pass][1][wave] = last;
    }
    __syncthreads();
    // (the target is the mass itself if u = 1 or by a rounding: the last that has any)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hit = min(i ? hit : INT32_MAX, found[pass][0][i]);
      last = max(last, found[pass][1][i]);
    }
    if (hit == INT32_MAX) hit = last;
    if (pass) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j == hit) {
          a.token[row] = hit;
          a.lp[row] = (float)(((double)v[j] - (double)st.max) / st.r.T - log(Z));
        }
    } else {
      seg = hit;
      // what lies before the segment comes off the target
      if (hit / 2 == (int)threadIdx.x) mass[0][0] = hit & 1 ? first + e[0] : first;
      __syncthreads();
      target -= mass[0][0];
    }
  }
}

// Rows of any class: one block of 1024 threads per row.
template <typename T>
__global__ void __launch_bounds__(1024) k_sample_pick(SampleArgs a) {
  __shared__ Lds l;
  const int64_t row = blockIdx.x;
  const int V = a.V, lane = threadIdx.x & 63, seg_of = threadIdx.x;
  const T* x = (const T*)a.logits + row * a.stride;
  RowState st;
  st.r = row_params(a, row);
  const RowRange range = row_range(a, row, l.range);
  st.max = range.top;
  if (!drawable(range, st.r)) {
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      a.lp[row] = __builtin_nanf("");
    }
    return;
  }

  // the row's whole mass, for lp; segment i belongs to thread i
  const bool has = seg_of < a.segs;
  double Z, s = 0.0;
  if (st.r.cls != NUCLEUS) {
    const double sum = has ? a.seg_sum[row * a.segs + seg_of] : 0.0;
    if (sum > 0.0) s = sum * st.weight(a.seg_max[row * a.segs + seg_of]);
  } else if (seg_of < a.splits) {
    s = a.z_part[row * a.splits + seg_of];
  }
  double at = block_before<double>(s, l.wave_d, Z), sum = Z;
  uint64_t cut = 0;
  RowClass cls = st.r.cls;
  if (cls != PLAIN) {
    if (seg_of < kMaxSegs) l.segs_u[seg_of] = cls == NUCLEUS && has ? a.seg_kept[row * a.segs + seg_of] : 0;
    if (cls == NUCLEUS) {
      const int n = a.listed[row];
      if (n <= kList) {
        for (int i = threadIdx.x; i < n; i += 1024) l.list[i] = a.list[row * kList + i];
        cut = cut_list(st, n, a.above[row], a.whole[row], l);
      } else {
        cls = GENERAL;
      }
    } else if (cls == LIST || cls == MIN_P) {
      const int n = candidates<T>(a, row, x, st, range.low, l);
      if (n <= kList) cut = cut_list(st, n, 0, 0, l);
      else cls = GENERAL;
    }
    if (__builtin_expect(cls == GENERAL, 0)) {
      if (st.r.k != 0) cut = find_cut<T, false>(x, V, st, 0, (uint64_t)st.r.k, 0.0, l);
      if (st.r.p != 0.0) {
        // the mass of what top-k keeps, exactly
        uint64_t part = 0, zk;
        for (int c = threadIdx.x * 8; c < V; c += 1024 * 8) {
          float v[8];
          load8(x, c, V, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < V && place(v[j], c + j) >= cut) part += units(st.weight(v[j]));
        }
        block_before<uint64_t>(part, l.wave_u, zk);
        const uint64_t c2 = find_cut<T, true>(x, V, st, cut, 0, st.r.p * (double)zk, l);
        cut = c2 > cut ? c2 : cut;
      }
      // the kept mass of each segment, one wave a segment
      for (int g = threadIdx.x >> 6; g < a.segs; g += 16) {
        uint64_t part = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = g * kSeg + q * 512 + lane * 8;
          float v[8];
          load8(x, c, V, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (c + j >= V || place(v[j], c + j) < cut) continue;
            const double e = st.weight(v[j]);
            if (e >= st.r.min_p) part += units(e);
          }
        }
        part = wave_total(part);
        if (lane == 0) l.segs_u[g] = part;
      }
      __syncthreads();
    }
    // at most 2^11 weights of at most 2^42 units: exact as a double
    s = has ? (double)l.segs_u[seg_of] * 0x1p-42 : 0.0;
    at = block_before<double>(s, l.wave_d, sum);
  }

  const double target = fmin(fmax((double)a.u[row], 0.0), 1.0) * sum;
  // the lowest segment whose running mass exceeds the target, else the last that has any
  // (the target is the mass itself if u = 1 or by a rounding)
  const int wave = threadIdx.x >> 6;
  int hit = s > 0.0 && at + s > target ? seg_of : INT32_MAX, end = s > 0.0 ? seg_of : -1;
  first_and_last(hit, end);
  if (lane == 0) {
    l.first[wave] = hit;
    l.last[wave] = end;
  }
  __syncthreads();
  hit = INT32_MAX;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    hit = min(hit, l.first[i]);
    end = max(end, l.last[i]);
  }
  const int seg = hit != INT32_MAX ? hit : end;
  if (seg_of == seg) l.wave_d[0] = at;
  __syncthreads();
  const double rest = target - l.wave_d[0];
  // its tokens, two a thread
  const int c = seg * kSeg + 2 * (int)threadIdx.x;
  float v[2];
  double e[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    v[j] = c + j < V ? (float)x[c + j] + 0.f : -__builtin_huge_valf();
    e[j] = v[j] > -__builtin_huge_valf() ? st.weight(v[j]) : 0.0;
    if (st.r.cls != PLAIN)
      e[j] = c + j < V && place(v[j], c + j) >= cut && e[j] >= st.r.min_p ? (double)units(e[j]) * 0x1p-42 : 0.0;
  }
  double run = block_before<double>(e[0] + e[1], l.wave_d, sum);
  hit = INT32_MAX, end = -1;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    run += e[j];
    if (e[j] > 0.0) {
      if (run > rest) hit = min(hit, c + j);
      end = c + j;
    }
  }
  first_and_last(hit, end);
  if (lane == 0) {
    l.first[wave] = hit;
    l.last[wave] = end;
  }
  __syncthreads();
  hit = INT32_MAX;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    hit = min(hit, l.first[i]);
    end = max(end, l.last[i]);
  }
  if (hit == INT32_MAX) hit = end;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (c + j == hit) {
      a.token[row] = hit;
      a.lp[row] = (float)(((double)v[j] - (double)st.max) / st.r.T - log(Z));
    }
}

struct SamplePlan {
  int64_t rows;          // per launch
  int segs, splits;
  size_t o_max, o_min, o_sum, o_grp, o_hist, o_z, o_above, o_whole, o_kept, o_listed, o_list, total;
};
// Rows go in batches, so that the workspace stays bounded; a row of at most kList tokens needs
// no histogram.  Splits: up to four blocks of 1024 threads per CU (rows of other classes leave theirs
// at once), each with at least 4 segments.
SamplePlan plan_sample(int64_t B, int64_t V) {
  SamplePlan p{};
  const bool nucleus = V > kList;
  p.rows = std::min<int64_t>(B, nucleus ? 1024 : 65536);
  p.segs = (int)((V + kSeg - 1) / kSeg);
  p.splits = nucleus ? (int)std::max<int64_t>(1, std::min<int64_t>((p.segs + 3) / 4, 1024 / p.rows)) : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes);
    return o;
  };
  const size_t n = (size_t)(p.rows * p.segs), h = (size_t)(p.rows * p.splits);
  p.o_max = take(n * 4);
  p.o_min = take(n * 4);
  p.o_sum = take(n * 8);
  p.o_grp = take(n * 256);
  p.o_hist = take(h * kNucleusBins * 8);
  p.o_z = take(h * 8);
  p.o_above = take((size_t)p.rows * 8);
  p.o_whole = take((size_t)p.rows * 8);
  p.o_kept = take(nucleus ? n * 8 : 0);
  p.o_listed = take((size_t)p.rows * 4);
  p.o_list = take(nucleus ? (size_t)p.rows * kList * 8 : 0);
  p.total = off;
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
hipError_t launch_sample(const SampleArgs& a, int64_t rows, hipStream_t s) {
  hipError_t e;
  {
    ScopedKernelTimer t(KK_SAMPLE_MASS, s);
    const int64_t waves = rows * a.segs;
    const int64_t blocks = std::min<int64_t>((waves + 3) / 4, 4 * kCUs);
    k_sample_mass<T><<<(unsigned)blocks, 256, 0, s>>>(a, waves);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // the two passes of NUCLEUS, where a row may be of that class
  if (a.V > kList && (a.p_rows != nullptr || (a.p > 0.0 && a.p < 1.0)) &&
      (a.k_rows != nullptr || a.k == 0 || a.k >= a.V)) {
    ScopedKernelTimer t(KK_SAMPLE_CUT, s);
    const dim3 grid((unsigned)a.splits, (unsigned)rows);
    k_sample_hist<T><<<grid, 1024, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    k_sample_gather<T><<<grid, 1024, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  ScopedKernelTimer t(KK_SAMPLE_PICK, s);
  const bool plain = a.k_rows == nullptr && a.p_rows == nullptr && a.min_p_rows == nullptr &&
                     (a.k == 0 || a.k >= a.V) && !(a.p > 0.0 && a.p < 1.0) && !(a.min_p > 0.0);
  if (plain) k_sample_plain<T><<<(unsigned)rows, 256, 0, s>>>(a);
  else k_sample_pick<T><<<(unsigned)rows, 1024, 0, s>>>(a);
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
  char* ws = (char*)workspace;
  hipStream_t s = (hipStream_t)stream;
  for (int64_t b = 0; b < B; b += p.rows) {
    const auto off = [b](auto* rows) { return rows == nullptr ? nullptr : rows + b; };
    grpo::SampleArgs a{};
    a.logits = (const char*)logits + b * row_stride * (dtype == GRPO_BF16 ? 2 : 4);
    a.u = u + b;
    a.stride = row_stride;
    a.V = (int)V;
    a.segs = p.segs;
    a.splits = p.splits;
    a.T = o.temperature;
    a.k = o.top_k;
    a.p = o.top_p;
    a.min_p = o.min_p;
    a.T_rows = off(o.temperature_rows);
    a.k_rows = off(o.top_k_rows);
    a.p_rows = off(o.top_p_rows);
    a.min_p_rows = off(o.min_p_rows);
    a.seg_max = (float*)(ws + p.o_max);
    a.seg_min = (float*)(ws + p.o_min);
    a.seg_sum = (double*)(ws + p.o_sum);
    a.grp_max = (float*)(ws + p.o_grp);
    a.hist = (uint64_t*)(ws + p.o_hist);
    a.z_part = (double*)(ws + p.o_z);
    a.above = (uint64_t*)(ws + p.o_above);
    a.whole = (uint64_t*)(ws + p.o_whole);
    a.seg_kept = (uint64_t*)(ws + p.o_kept);
    a.listed = (int*)(ws + p.o_listed);
    a.list = (uint64_t*)(ws + p.o_list);
    a.token = token + b;
    a.lp = lp + b;
    const int64_t rows = std::min(p.rows, B - b);
    GRPO_HIP(dtype == GRPO_BF16 ? grpo::launch_sample<__bf16>(a, rows, s)
                                : grpo::launch_sample<float>(a, rows, s));
  }
  return GRPO_OK;
}

}  // extern "C"
