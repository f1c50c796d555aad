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
// 2^20 tokens are exact in 64 bits: no result depends on an order.  Each weight of a filtered row is
// so rounded by up to 2^-43 of the heaviest one's: what lies 30 T below the maximum weighs nothing
// there, and 10^5 such tokens lose up to 10^-8 of the mass.
//
// Rows by what their filters need, each with the fewest passes over the logits:
//   PLAIN   no filter: one pass for maxima and sums, then one segment of 2048 tokens.
//   LIST    top-k up to 2048, with or without the others, or any filter on a row of at most
//           4096: the first pass keeps the maximum of every 32 tokens; at least k of these
//           are at or above the k-th largest of them, so every kept token is, and only the
//           groups whose maximum is are read again.  The cuts are found among those candidates.
//   MIN_P   min-p alone: one more pass over the segments whose maximum reaches min_p.
//   HIST    top-p, alone or with a larger k: histograms of mass and count over 2048 or 4096 bins of x
//           tell which bins the cuts fall into; one more pass sums what lies above them and
//           lists the tokens of those bins, among which the cuts are found.
// Lists hold up to 4096 tokens; where one overflows, the cuts are found among all tokens of the row,
// by the same search in up to five passes of one block.  Equal logits do that, and finite masks where
// LIST's bins reach from the maximum to the least group's or HIST's, with a k, to the row's minimum:
// -1e9 in 267 of 151936 tokens leaves all the others in one bin.  64 such rows with top-k 50 take
// 320 us, with top-p as well 510 us; with -inf there 31 and 32 us.
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
constexpr int kHistThreads = 512;
// Bins of HIST: 2048 keep the passes over them short; a flat row of 2^18 tokens then has some 2000
// in its fullest bin.  4096 for longer rows.
constexpr int64_t kFewBins = 1 << 18;
constexpr int hist_bins_for(int64_t V) { return V <= kFewBins ? 2048 : 4096; }
constexpr int kBins = 2048;                // of the groups' maxima, and of one pass of a search
constexpr int kList = 4096;                // listed tokens of a row
constexpr int kListK = 2048;               // largest top-k that goes by the groups' maxima
constexpr int kPick = 256;                 // threads of a row's last step
constexpr int kLine = 32;                  // integers of a 128-byte line
constexpr float kNone = -__builtin_huge_valf();

// What HIST's gather and pick need to know: tokens in bins below `sure` are kept (but for
// min-p); those of bins lo .. hi and of bin kbin are listed.  The offsets make ranks and running
// masses among the listed tokens those among all that matter: see k_sample_cut.
struct RowCut {
  int sure, lo, hi, kbin;
  int k;                 // 0: no k, or fewer tokens than k
  float top, low;        // the row's range; NaN: nothing to draw from
  int pad;
  uint64_t count_off, mass_off, z_off;
};

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
  float* seg_min;      // [B, segs], of what is above -inf: HIST all tokens, LIST the groups' maxima
  double* seg_sum;     // [B, segs], relative to the segment's own maximum (not for HIST)
  float* grp_max;      // [B, segs, 64]: a lane's 32 tokens (LIST)
  uint64_t* seg_kept;  // [B, segs]: mass that is surely kept (HIST, MIN_P)
  int* listed;         // [B, kLine]: tokens in the list, each row's number in a cache line of its own
  // HIST
  uint64_t* hist;      // [B, splits, bins]: masses
  uint32_t* hist_n;    // [B, splits, bins]: counts
  double* z_part;      // [B, splits]
  RowCut* cut;         // [B]
  uint64_t* list;      // [B, kList]: places
  int32_t* token;
  float* lp;
};

enum RowClass { PLAIN, LIST, MIN_P, HIST };

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
  else r.cls = r.k != 0 || r.p != 0.0 ? HIST : MIN_P;
  return r;
}

// 2^t for t <= 0: t = n + f with n whole and |f| <= 1/2, and 2^f by the polynomial 1 + f q(f) of
// degree 9 whose largest relative error is the least one, below 1.6e-14 (with 10^5 borders in a
// row, one row in 10^8 has u that near one).  It is off by the same at both ends, -1.51e-14, so that
// weights do not jump from one n to the next.  Below 2^-1000 it stays at 2^-1000, which adds nothing
// to a sum beside the row's maximum, whose weight is 1; where a token is drawn it counts as 0
// (RowState::mass).
__device__ __forceinline__ double pow2_down(double t) {
  t = fmax(t, -1000.0);
  const double magic = 0x1.8p52, shifted = t + magic;
  const double f = t - (shifted - magic);
  double q = 0x1.b3de31389fe36p-24;
  q = fma(q, f, 0x1.63e6964c004b3p-20);
  q = fma(q, f, 0x1.ffce2fc0b9a32p-17);
  q = fma(q, f, 0x1.430897f348181p-13);
  q = fma(q, f, 0x1.5d87fd938895cp-10);
  q = fma(q, f, 0x1.3b2ab72412178p-7);
  q = fma(q, f, 0x1.c6b08d70c880dp-5);
  q = fma(q, f, 0x1.ebfbdff81be06p-3);
  q = fma(q, f, 0x1.62e42fefa37d1p-1);
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
// One wave per segment of one row: 28 instructions a token, most of them float64, against
// 4 bytes: 256 x 128256 in float32 take 34 us, of which the loads alone need 27.  (Waves that walk
// over segments and load the next one ahead took 37: more of them at once hide more.)
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
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < waves; w += (int64_t)gridDim.x * 4) {
    const RawSeg<T> raw = load_seg<T>(a, w / a.segs, (int)(w % a.segs));
    float x[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[q][j] = (float)raw.q[q].v[j / kVec<T>][j % kVec<T>];
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
    low = m > kNone ? m : __builtin_huge_valf();
    if (r.cls == LIST) a.grp_max[w * 64 + lane] = m;
    if (r.cls == HIST) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[q][j] > kNone) low = fminf(low, x[q][j]);
    }
    if (r.cls != PLAIN) low = wave_low(low);
    m = wave_top(m);
    const bool bad = __any(nan) || m == __builtin_huge_valf();
    double s = 0.0;
    if (r.cls != HIST && m > kNone) {
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
      if (w % a.segs == 0) a.listed[w / a.segs * kLine] = 0;
    }
  }
}

// ---------------------------------------------------------------- the order
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
  // The weight, 0 below 2^-1000: what the pick may draw for u = 0 or 1 must not be what a finite
  // mask or a temperature near zero leaves.  (The sums go without the test: it would be two more
  // instructions for each token of k_sample_mass, whose sums it does not change.)
  __device__ __forceinline__ double mass(float x) const {
    const double t = ((double)x - (double)max) * r.rate;
    return t < -1000.0 ? 0.0 : pow2_down(t);
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

// Sums over a block of NT threads of the values before this thread's, and the total.
template <int NT, typename V>
__device__ __forceinline__ V block_before(V v, V* lds, V& total) {
  V wt;
  const V before = wave_before(v, wt);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = wt;
  __syncthreads();
  V off = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    if (i < (int)(threadIdx.x >> 6)) off += lds[i];
    total += lds[i];
  }
  return off + before;
}

// A row's maximum over its segments, whether it holds a NaN or +inf, and the least of the
// segments' minima, from each thread's share of them (lds: 3 for each wave).
struct RowRange {
  float top, low;
  bool bad;
};
template <int NT>
__device__ __forceinline__ RowRange row_range(float top, float low, bool bad, float (*lds)[NT / 64]) {
  RowRange r{wave_top(top), wave_low(low), (bool)__any(bad)};
  if ((threadIdx.x & 63) == 0) {
    const int w = threadIdx.x >> 6;
    lds[0][w] = r.top;
    lds[1][w] = r.low;
    lds[2][w] = r.bad ? 1.f : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    r.top = fmaxf(r.top, lds[0][w]);
    r.low = fminf(r.low, lds[1][w]);
    r.bad |= lds[2][w] != 0.f;
  }
  return r;
}
template <int NT>
__device__ __forceinline__ RowRange row_range(const SampleArgs& a, int64_t row, float (*lds)[NT / 64]) {
  float top = kNone, low = -kNone;
  bool bad = false;
  // a thread past the last segment looks at the last one again
#pragma unroll
  for (int i = 0; i < kMaxSegs; i += NT) {
    const int64_t at = row * a.segs + min(i + (int)threadIdx.x, a.segs - 1);
    const float m = a.seg_max[at];
    top = fmaxf(top, m);
    bad |= m != m;
    low = fminf(low, a.seg_min[at]);
  }
  return row_range<NT>(top, low, bad, lds);
}
// Whether there is anything to draw from.
__device__ __forceinline__ bool drawable(const RowRange& g, const RowParams& r) {
  return !g.bad && g.top > kNone && r.T > 0.0 && r.T < __builtin_huge_val();
}
// Over 30 T below the maximum, 2^20 tokens weigh less than 10^-6 of it.  With a k, the bins go
// down to the minimum: tokens without weight count too.
__device__ __forceinline__ Binning hist_bins(const RowRange& g, const RowParams& r, int bins) {
  const float all = g.top - g.low;
  return Binning(g.top, r.k != 0 ? all : fminf(all, (float)(30.0 * r.T)), bins);
}

// ---------------------------------------------------------------- HIST
// Block (split, row): the mass and number of the split's tokens by bin.
template <typename T, int BINS>
__global__ void __launch_bounds__(kHistThreads) k_sample_hist(SampleArgs a) {
  constexpr int NT = kHistThreads;
  const int64_t row = blockIdx.y;
  RowState st;
  st.r = row_params(a, row);
  if (st.r.cls != HIST) return;
  __shared__ uint64_t mass[BINS];
  __shared__ uint32_t number[BINS];
  __shared__ float range[3][NT / 64];
  __shared__ double zs[NT / 64];
  const int per = (a.segs + a.splits - 1) / a.splits * kSeg;
  const int from = min(a.V, (int)blockIdx.x * per), to = min(a.V, from + per);
  const T* x = (const T*)a.logits + row * a.stride;
  Raw8<T> next = {};
  if (from + (int)threadIdx.x * 8 < to) next = load8(x, from + threadIdx.x * 8, a.V);
  for (int i = threadIdx.x; i < BINS; i += NT) mass[i] = number[i] = 0;
  const RowRange g = row_range<NT>(a, row, range);      // its barrier is also the bins'
  if (!drawable(g, st.r)) return;
  st.max = g.top;
  const Binning bin = hist_bins(g, st.r, BINS);
  const bool counted = st.r.k != 0;
  double z = 0.0;
  for (int c = from + threadIdx.x * 8; c < to; c += NT * 8) {
    float v[8];
    unpack(next, v);
    if (c + NT * 8 < to) next = load8(x, c + NT * 8, a.V);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double e = st.weight(v[j]);
      const uint64_t n = units(e);
      const int b = bin(v[j]);
      z += e;
      if (n) atomicAdd((unsigned long long*)&mass[b], (unsigned long long)n);
      if (counted && v[j] > kNone) atomicAdd(&number[b], 1u);
    }
  }
  double total;
  block_before<NT, double>(z, zs, total);
  const int64_t at = (row * a.splits + blockIdx.x) * BINS;
  for (int i = threadIdx.x; i < BINS; i += NT) {
    a.hist[at + i] = mass[i];
    if (counted) a.hist_n[at + i] = number[i];
  }
  if (threadIdx.x == 0) a.z_part[row * a.splits + blockIdx.x] = total;

}

// One block per row: adds the splits up and finds the bins of the cuts.  (The last block of a row
// could do it in k_sample_hist, but its release fence writes back the whole L2: 200 us.)
//
// Let kbin be the bin of the k-th token, and lo .. hi the bins in which the share p of the mass
// may be reached: it is of the mass of the first k, which lies between that above kbin and that
// with kbin.  Listed are bins lo .. hi and kbin.  Among the listed tokens, in their order:
//   rank + count_off   is the rank among all for those of kbin, and less for the others;
//   mass + mass_off    is the mass before among all for those of lo .. hi, and at least the
//                      share for those of kbin behind them;
//   z_off + the mass of the listed ones up to rank k is that of the first k of all.
template <int BINS>
__global__ void __launch_bounds__(kHistThreads) k_sample_cut(SampleArgs a) {
  constexpr int NT = kHistThreads, PER = BINS / NT;
  const int64_t row = blockIdx.x;
  RowState st;
  st.r = row_params(a, row);
  if (st.r.cls != HIST) return;
  __shared__ float range[3][NT / 64];
  __shared__ uint64_t sums[NT / 64];
  __shared__ RowCut rc;
  __shared__ uint64_t above_k, with_k;
  const bool counted = st.r.k != 0;
  const RowRange g = row_range<NT>(a, row, range);
  if (!drawable(g, st.r)) {
    if (threadIdx.x == 0) a.cut[row].top = __builtin_nanf("");
    return;
  }
  // thread t holds bins PER t ..
  uint64_t h[PER], own = 0, whole;
  uint32_t n[PER], own_n = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) h[j] = n[j] = 0;
  // 8 splits' loads at a time
  for (int s0 = 0; s0 < a.splits; s0 += 8) {
    typedef __attribute__((ext_vector_type(2))) uint64_t U2;
    typedef __attribute__((ext_vector_type(4))) uint32_t U4;
    U2 in[8][PER / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < PER / 2; ++j)
        in[i][j] = s0 + i < a.splits
                       ? ((const U2*)(a.hist + (row * a.splits + s0 + i) * BINS))[PER / 2 * threadIdx.x + j]
                       : U2{0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < PER; ++j) h[j] += in[i][j / 2][j % 2];
    if (counted) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < PER / 4; ++j)
          if (s0 + i < a.splits) {
            const U4 in_n = ((const U4*)(a.hist_n + (row * a.splits + s0 + i) * BINS))[PER / 4 * threadIdx.x + j];
#pragma unroll
            for (int q = 0; q < 4; ++q) n[4 * j + q] += in_n[q];
          }
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    own += h[j];
    own_n += n[j];
  }
  if (threadIdx.x == 0) rc = RowCut{0, 1, 0, -1, 0, g.top, g.low, 0, 0, 0, 0};
  const uint64_t first = block_before<NT, uint64_t>(own, sums, whole);
  uint64_t n_all, n_run = 0, k = (uint64_t)st.r.k;
  if (counted) {
    n_run = block_before<NT, uint64_t>(own_n, sums, n_all);
    uint64_t run = first;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (n_run < k && n_run + n[j] >= k) {          // one thread's, if any
        rc.kbin = rc.sure = PER * threadIdx.x + j;
        rc.k = st.r.k;
        rc.count_off = n_run;
        above_k = run;
        with_k = run + h[j];
      }
      n_run += n[j];
      run += h[j];
    }
    __syncthreads();
  }
  const int kbin = rc.kbin;                          // -1: no k, or fewer tokens than k
  if (kbin < 0 && st.r.p == 0.0 && threadIdx.x == 0) rc.sure = BINS;    // then all are kept
  if (st.r.p != 0.0) {
    const double least = st.r.p * (double)(kbin >= 0 ? above_k : whole);
    const double most = st.r.p * (double)(kbin >= 0 ? with_k : whole);
    uint64_t run = first;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (h[j] && (double)run < most && (double)(run + h[j]) >= most) rc.hi = PER * threadIdx.x + j;
      if (h[j] && (double)run < least && (double)(run + h[j]) >= least) {
        rc.lo = rc.sure = PER * threadIdx.x + j;
        rc.mass_off = run;
      }
      run += h[j];
    }
    if (threadIdx.x == 0 && !(least > 0.0)) rc.lo = rc.sure = 0, rc.mass_off = 0;
    __syncthreads();
    // what is listed but for kbin
    uint64_t listed = 0, listed_n = 0, sum, sum_n;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int b = PER * threadIdx.x + j;
      if (b >= rc.lo && b <= rc.hi && b != kbin) {
        listed += h[j];
        listed_n += n[j];
      }
    }
    block_before<NT, uint64_t>(listed, sums, sum);
    block_before<NT, uint64_t>(listed_n, sums, sum_n);
    if (threadIdx.x == 0) {
      rc.z_off = (kbin >= 0 ? above_k : whole) - sum;
      if (kbin >= 0) rc.count_off -= sum_n;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.cut[row] = rc;
}

// Block (four segments, row) of HIST and MIN_P: the surely kept mass of each segment and the
// list of what is not sure.  Segments whose maximum is below both are left out.
template <typename T>
__global__ void __launch_bounds__(256) k_sample_gather(SampleArgs a) {
  const int64_t row = blockIdx.y;
  RowState st;
  st.r = row_params(a, row);
  if (st.r.cls != HIST && st.r.cls != MIN_P) return;
  __shared__ float range[3][4];
  __shared__ int counts[4], first;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int seg = min(a.segs - 1, (int)blockIdx.x * 4 + wave);
  const float top = a.seg_max[row * a.segs + seg];
  RowCut rc{INT32_MAX, 1, 0, -1, 0, 0.f, 0.f, 0, 0, 0, 0};
  if (st.r.cls == HIST) rc = a.cut[row];
  const RawSeg<T> raw = load_seg<T>(a, row, seg);       // on its way while the row's range is found
  RowRange g{rc.top, rc.low, rc.top != rc.top};
  if (st.r.cls == MIN_P) g = row_range<256>(a, row, range);
  if (!drawable(g, st.r)) return;
  st.max = g.top;
  const int bins = hist_bins_for(a.V);
  Binning bin(g.top, 0.f, bins);
  bool read = st.weight(top) >= st.r.min_p;
  if (st.r.cls == HIST) {
    bin = hist_bins(g, st.r, bins);
    const int b = bin(top);
    read = b < rc.sure || b <= rc.hi || b <= rc.kbin;
  }
  const bool own = (int)blockIdx.x * 4 + wave < a.segs;
  uint64_t part = 0;
  unsigned unsure = 0;
  if (read && own) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8];
      unpack(raw.q[q], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int b = bin(v[j]);
        if (b < rc.sure) {
          const double e = st.weight(v[j]);
          if (e >= st.r.min_p) part += units(e);
        }
        if (((b >= rc.lo && b <= rc.hi) || b == rc.kbin) && v[j] > kNone) unsure |= 1u << (q * 8 + j);
      }
    }
    part = wave_total(part);
  }
  if (lane == 0 && own) a.seg_kept[row * a.segs + seg] = part;
  if (st.r.cls != HIST) return;
  // one addition to the row's number for the block
  int all, slot = wave_before((int)__popc(unsure), all);
  if (lane == 0) counts[wave] = all;
  __syncthreads();
  if (threadIdx.x == 0) {
    const int sum = counts[0] + counts[1] + counts[2] + counts[3];
    first = sum ? atomicAdd(&a.listed[row * kLine], sum) : 0;
  }
  __syncthreads();
  if (all == 0) return;
  slot += first;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < wave) slot += counts[i];
  // more than kList in all: the pick sees the number and goes by the row
  const int c0 = seg * kSeg + lane * 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
    unpack(raw.q[q], v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((unsure >> (q * 8 + j)) & 1) {
        if (slot < kList) a.list[row * kList + slot] = place(v[j], c0 + q * 512 + j);
        ++slot;
      }
  }
}

// ---------------------------------------------------------------- the pick
struct Lds {
  uint64_t list[kList];
  union {
    uint64_t bins[kBins];
    uint32_t counts[kBins];
    int groups[2 * kBins];
  };
  uint64_t segs[kMaxSegs];
  uint64_t wave_u[kPick / 64];
  uint64_t found_sum, result;
  int found, count;
};

// The place, in [lo, hi], of the token with which the running count (or mass, in units) reaches
// `target`, in order from the top, `base` of it lying above hi; lo if it does not.  each(f) calls
// f for the place of every token.  Passes over ever smaller ranges, of 2048 bins each, until 256
// tokens are left, which are compared directly.
template <bool MASS, typename Each>
__device__ __forceinline__ uint64_t search(const Each& each, uint64_t lo, uint64_t hi, uint64_t base,
                                           double target, const RowState& st, Lds& l) {
  const auto amount = [&](uint64_t p) { return MASS ? units(st.weight(value_at(p))) : (uint64_t)1; };
  const auto reached = [&](uint64_t sum) { return (double)sum >= target; };
  for (;;) {
    const uint64_t span = hi - lo;
    const int shift = span < kBins ? 0 : 64 - __clzll((long long)span) - 11;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBins / kPick; ++i) l.bins[threadIdx.x + i * kPick] = 0;
    if (threadIdx.x == 0) {
      l.found = -1;
      l.count = 0;
    }
    __syncthreads();
    each([&](uint64_t p) {
      if (p < lo || p > hi) return;
      const uint64_t n = amount(p);
      if (n) atomicAdd((unsigned long long*)&l.bins[(hi - p) >> shift], (unsigned long long)n);
    });
    __syncthreads();
    constexpr int PER = kBins / kPick;
    uint64_t h[PER], own = 0, total;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      h[j] = l.bins[PER * threadIdx.x + j];
      own += h[j];
    }
    uint64_t run = base + block_before<kPick, uint64_t>(own, l.wave_u, total);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (h[j] && !reached(run) && reached(run + h[j])) {
        l.found = PER * threadIdx.x + j;
        l.found_sum = run;
      }
      run += h[j];
    }
    __syncthreads();
    if (l.found < 0) return lo;
    base = l.found_sum;
    hi -= (uint64_t)l.found << shift;
    const uint64_t rest = ((uint64_t)1 << shift) - 1;
    if (hi - lo > rest) lo = hi - rest;
    if (lo == hi) return lo;
    // the bin's tokens, if they are few
    each([&](uint64_t p) {
      if (p < lo || p > hi) return;
      const int slot = atomicAdd(&l.count, 1);
      if (slot < kPick) l.bins[slot] = p;
    });
    __syncthreads();
    const int n = l.count;
    if (n > kPick) continue;
    const int t = threadIdx.x;
    const uint64_t p = t < n ? l.bins[t] : 0, mine = t < n ? amount(p) : 0;
    if (t < n) l.bins[kPick + t] = mine;
    __syncthreads();
    uint64_t before = base;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const uint64_t other = l.bins[i], amount = l.bins[kPick + i];
      before += other > p ? amount : 0;
    }
    if (mine && !reached(before) && reached(before + mine)) l.result = p;
    __syncthreads();
    return l.result;
  }
}

// The place of the last kept token among n tokens that each(f) goes through, with the offsets of
// RowCut; 0 for none (a row with fewer tokens than k: no cut).  Up to 256 of them (the usual top-k)
// are compared directly: each thread ranks one.
template <typename Each>
__device__ __forceinline__ uint64_t last_kept(const Each& each, int n, const RowCut& rc, const RowState& st,
                                              Lds& l) {
  const int t = threadIdx.x;
  const uint64_t k = rc.k != 0 ? (uint64_t)rc.k : ~(uint64_t)0;
  if (n == 0) return 0;
  if (n <= kPick) {
    const uint64_t p = t < n ? l.list[t] : 0, mine = t < n ? units(st.weight(value_at(p))) : 0;
    if (t < n) l.bins[t] = mine;
    if (t == 0) l.result = ~(uint64_t)0;
    __syncthreads();
    uint64_t rank = rc.count_off, before = rc.mass_off, first_k;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const uint64_t other = l.list[i], amount = l.bins[i];
      rank += other > p ? 1 : 0;
      before += other > p ? amount : 0;
    }
    bool keep = t < n && rank < k;
    if (st.r.p != 0.0) {
      block_before<kPick, uint64_t>(keep ? mine : 0, l.wave_u, first_k);
      keep = keep && (double)before < st.r.p * (double)(rc.z_off + first_k);
    }
    // the least of the kept places: one lane a wave
    uint64_t least = keep ? p : ~(uint64_t)0;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const uint64_t other = __shfl_xor((unsigned long long)least, o, 64);
      least = other < least ? other : least;
    }
    if ((t & 63) == 0) atomicMin((unsigned long long*)&l.result, (unsigned long long)least);
    __syncthreads();
    return l.result;
  }
  // the range of the places
  uint64_t top = 0, low = ~(uint64_t)0;
  each([&](uint64_t p) {
    top = p > top ? p : top;
    low = p < low ? p : low;
  });
  if (t == 0) {
    l.result = 0;
    l.found_sum = ~(uint64_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint64_t high = __shfl_xor((unsigned long long)top, o, 64), deep = __shfl_xor((unsigned long long)low, o, 64);
    top = high > top ? high : top;
    low = deep < low ? deep : low;
  }
  if ((t & 63) == 0) {
    atomicMax((unsigned long long*)&l.result, (unsigned long long)top);
    atomicMin((unsigned long long*)&l.found_sum, (unsigned long long)low);
  }
  __syncthreads();
  top = l.result;
  low = l.found_sum;
  uint64_t cut = low;
  if (rc.k != 0) cut = search<false>(each, low, top, rc.count_off, (double)k, st, l);
  if (st.r.p != 0.0) {
    uint64_t sum = 0, first_k;
    each([&](uint64_t p) {
      if (p >= cut) sum += units(st.weight(value_at(p)));
    });
    block_before<kPick, uint64_t>(sum, l.wave_u, first_k);
    cut = search<true>(each, cut, top, rc.mass_off, st.r.p * (double)(rc.z_off + first_k), st, l);
  }
  return cut;
}

// LIST: the tokens that may be kept, into l.list; their number (over kList: too many).  A group
// is 32 tokens that one lane of k_sample_mass read; only groups whose maximum may be kept are
// read again.  `low`: the least of the groups' maxima.
template <typename T>
__device__ __forceinline__ int candidates(const SampleArgs& a, int64_t row, const T* x,
                                          const RowState& st, float low, Lds& l) {
  const int groups = a.segs * 64, lane = threadIdx.x & 63;
  const float* gm = a.grp_max + row * groups;
  // 8192 groups at a time, in registers: thread t holds groups 256 i + t
  constexpr int HELD = 32;
  float g[HELD];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int at = base + i * kPick + (int)threadIdx.x;
      g[i] = gm[min(at, groups - 1)];
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (base + i * kPick + (int)threadIdx.x >= groups) g[i] = kNone;
  };
  load(0);
  Binning bin(st.max, 0.f, kBins);          // all that is above -inf into bin 0
  int last = kBins - 1;
  __syncthreads();
  if (a.V > kList) {
    // bins over the range of the groups' maxima; the last one that the k largest reach into
    const Binning fine(st.max, st.max - low, kBins);
#pragma unroll
    for (int i = 0; i < kBins / kPick; ++i) l.counts[threadIdx.x + i * kPick] = 0;
    if (threadIdx.x == 0) l.found = -1;
    __syncthreads();
#pragma unroll 1
    for (int base = 0; base < groups; base += HELD * kPick) {
      if (base) load(base);
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (g[i] > kNone) atomicAdd(&l.counts[fine(g[i])], 1u);
    }
    __syncthreads();
    constexpr int PER = kBins / kPick;
    uint64_t c[PER], own = 0, total;
    const uint64_t k = (uint64_t)st.r.k;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      c[j] = l.counts[PER * threadIdx.x + j];
      own += c[j];
    }
    uint64_t run = block_before<kPick, uint64_t>(own, l.wave_u, total);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (run < k && run + c[j] >= k) l.found = PER * threadIdx.x + j;
      run += c[j];
    }
    __syncthreads();
    if (l.found >= 0) {                     // otherwise fewer groups than k: all of them
      last = l.found;
      bin = fine;
    }
    if (groups > HELD * kPick) load(0);
  }
  if (threadIdx.x == 0) l.count = l.found_sum = 0;
  __syncthreads();
  // the wanted groups: each has a token for the list, so that over kList of them are too many
  auto wanted = [&](float v) { return v > kNone && bin(v) <= last; };
  int* n_groups = (int*)&l.found_sum;
  // one slot for each set bit of every lane's mask: one LDS atomic a wave
  auto slots = [&](unsigned mask, int* counter) {
    int all, at = wave_before((int)__popc(mask), all), first = 0;
    if (all == 0) return 0;
    if (lane == 0) first = atomicAdd(counter, all);
    return at + __builtin_amdgcn_readfirstlane(first);
  };
#pragma unroll 1
  for (int base = 0; base < groups; base += HELD * kPick) {
    if (base) load(base);
    unsigned want = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) want |= wanted(g[i]) ? 1u << i : 0u;
    int at = slots(want, n_groups);
    for (; want; want &= want - 1, ++at)
      if (at < kList) l.groups[at] = base + (__ffs(want) - 1) * kPick + (int)threadIdx.x;
  }
  __syncthreads();
  const int wanted_groups = *n_groups;
  if (wanted_groups > kList) return kList + 1;
  // 32 threads to a group, 16 tokens of each thread at a time
  // (their loads are not under a condition: a branch for each would wait for it)
  constexpr int AT_ONCE = 16;
#pragma unroll 1
  for (int e0 = 0; e0 < wanted_groups * 32; e0 += kPick * AT_ONCE) {
    T v[AT_ONCE];
    int c[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int e = e0 + i * kPick + (int)threadIdx.x, r = e & 31;
      // tokens q * 512 + lane * 8 + j of the segment, q < 4 and j < 8
      const int id = l.groups[min(e >> 5, wanted_groups - 1)];
      c[i] = (id >> 6) * kSeg + (r >> 3) * 512 + (id & 63) * 8 + (r & 7);
      v[i] = x[min(c[i], a.V - 1)];
    }
    unsigned take = 0;
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const bool in = e0 + i * kPick + (int)threadIdx.x < wanted_groups * 32 && c[i] < a.V;
      take |= in && wanted((float)v[i] + 0.f) ? 1u << i : 0u;
    }
    int at = slots(take, &l.count);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if ((take >> i) & 1) {
        if (at < kList) l.list[at] = place((float)v[i] + 0.f, c[i]);
        ++at;
      }
  }
  __syncthreads();
  return l.count;
}

// One block of 256 threads per row: what is kept (not for PLAIN), then where the running mass
// first exceeds u times the kept mass, by segments and in the segment.  Its time is that of a
// chain of loads and barriers, so it has few waves; a kernel of its own serves calls without
// filters (4.9 us for a row of 151936 tokens; with top-k 50 and top-p 16).
template <typename T, bool FILTERED>
__global__ void __launch_bounds__(kPick) k_sample_pick(SampleArgs a) {
  struct Small {
    float range[3][kPick / 64];
    double mass[2][kPick / 64];
    int found[2][2][kPick / 64];
  };
  __shared__ Small sh;
  const int64_t row = blockIdx.x;
  const int V = a.V, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* x = (const T*)a.logits + row * a.stride;
  // thread t holds segments 2t and 2t + 1
  float m[2], low = -kNone;
  double s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t i = row * a.segs + min(2 * (int)threadIdx.x + j, a.segs - 1);
    m[j] = a.seg_max[i];
    s[j] = a.seg_sum[i];
    if (FILTERED) low = fminf(low, a.seg_min[i]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (2 * (int)threadIdx.x + j >= a.segs) {
      m[j] = kNone;
      s[j] = 0.0;
    }
  const double u = fmin(fmax((double)a.u[row], 0.0), 1.0);
  RowState st;
  st.r = row_params(a, row);
  const RowRange g = row_range<kPick>(fmaxf(m[0], m[1]), low, m[0] != m[0] || m[1] != m[1], sh.range);
  st.max = g.top;
  if (!drawable(g, st.r)) {
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      a.lp[row] = __builtin_nanf("");
    }
    return;
  }
  double e[8], Z = 0.0, target = 0.0;
#pragma unroll
  for (int j = 0; j < 2; ++j) e[j] = s[j] > 0.0 ? s[j] * st.mass(m[j]) : 0.0;
  uint64_t cut = 0;
  const bool filtered = FILTERED && st.r.cls != PLAIN;
  if constexpr (FILTERED) {
    __shared__ Lds l;
    if (filtered) {
      // the row's whole mass, for lp
      if (st.r.cls == HIST)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = 2 * threadIdx.x + j;
          e[j] = i < a.splits ? a.z_part[row * a.splits + i] : 0.0;
        }
      block_before<kPick, double>(e[0] + e[1], sh.mass[1], Z);
      const bool sure = st.r.cls != LIST;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * threadIdx.x + j;
        l.segs[i] = sure && i < a.segs ? a.seg_kept[row * a.segs + i] : 0;
      }
      if (st.r.cls != MIN_P) {
        RowCut rc{0, 0, 0, 0, st.r.k, 0.f, 0.f, 0, 0, 0, 0};
        int n;
        if (st.r.cls == LIST) {
          n = candidates<T>(a, row, x, st, g.low, l);
        } else {
          rc = a.cut[row];
          n = a.listed[row * kLine];
          if (n <= kList)
            for (int i = threadIdx.x; i < n; i += kPick) l.list[i] = a.list[row * kList + i];
          __syncthreads();
        }
        if (n <= kList) {
          const auto listed = [&](auto f) {
            for (int i = threadIdx.x; i < n; i += kPick) f(l.list[i]);
          };
          cut = last_kept(listed, n, rc, st, l);
          listed([&](uint64_t p) {
            const double w = st.weight(value_at(p));
            if (p >= cut && w >= st.r.min_p)
              atomicAdd((unsigned long long*)&l.segs[index_at(p) / kSeg], (unsigned long long)units(w));
          });
        } else {
          const auto all = [&](auto f) {
            for (int c = threadIdx.x * 8; c < V; c += kPick * 8) {
              float v[8];
              load8(x, c, V, v);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (v[j] > kNone) f(place(v[j], c + j));
            }
          };
          cut = last_kept(all, INT32_MAX, RowCut{0, 0, 0, 0, st.r.k, 0.f, 0.f, 0, 0, 0, 0}, st, l);
          __syncthreads();
#pragma unroll
          for (int j = 0; j < 2; ++j) l.segs[2 * threadIdx.x + j] = 0;
          __syncthreads();
          all([&](uint64_t p) {
            const double w = st.weight(value_at(p));
            if (p >= cut && w >= st.r.min_p)
              atomicAdd((unsigned long long*)&l.segs[index_at(p) / kSeg], (unsigned long long)units(w));
          });
        }
      }
      __syncthreads();
      // at most 2^11 weights of at most 2^42 units: exact as a double
#pragma unroll
      for (int j = 0; j < 2; ++j) e[j] = (double)l.segs[2 * threadIdx.x + j] * 0x1p-42;
    }
  }
  int seg = 0;
  float v[8];
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int c = pass ? seg * kSeg + (int)threadIdx.x * 8 : 2 * (int)threadIdx.x;
    if (pass) {
      load8(x, c, V, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = v[j] > kNone ? st.mass(v[j]) : 0.0;
        if (filtered)
          e[j] = v[j] > kNone && place(v[j], c + j) >= cut && e[j] >= st.r.min_p ? (double)units(e[j]) * 0x1p-42 : 0.0;
      }
    }
    double own = 0.0;
#pragma unroll
    for (int j = 0; j < (pass ? 8 : 2); ++j) own += e[j];
    double wt, sum = 0.0;
    double run = wave_before(own, wt);
    if (lane == 63) sh.mass[pass][wave] = wt;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPick / 64; ++i) {
      if (i < wave) run += sh.mass[pass][i];
      sum += sh.mass[pass][i];
    }
    if (!pass) {
      target = u * sum;
      if (!filtered) Z = sum;
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
      sh.found[pass][0][wave] = hit;
      sh.found[pass][1][wave] = last;
    }
    __syncthreads();
    // (the target is the mass itself if u = 1 or by a rounding: the last that has any)
#pragma unroll
    for (int i = 0; i < kPick / 64; ++i) {
      hit = min(i ? hit : INT32_MAX, sh.found[pass][0][i]);
      last = max(last, sh.found[pass][1][i]);
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
      seg = max(hit, 0);   // -1 only if another call writes the workspace meanwhile
      // what lies before the segment comes off the target
      if (hit / 2 == (int)threadIdx.x) sh.mass[0][0] = hit & 1 ? first + e[0] : first;
      __syncthreads();
      target -= sh.mass[0][0];
    }
  }
}

struct SamplePlan {
  int64_t rows;          // per launch
  int segs, splits;
  size_t o_max, o_min, o_sum, o_grp, o_kept, o_listed, o_hist, o_hist_n, o_z, o_cut, o_list, total;
};
// Rows go in batches, so that the workspace stays bounded; a row of at most kList tokens needs
// no histogram.  Splits: about three blocks of 512 threads per CU, each with at least 4 segments.
SamplePlan plan_sample(int64_t B, int64_t V) {
  SamplePlan p{};
  const bool hist = V > kList;
  p.rows = std::min<int64_t>(B, hist ? 1024 : 65536);
  p.segs = (int)((V + kSeg - 1) / kSeg);
  p.splits = hist ? (int)std::max<int64_t>(1, std::min<int64_t>((p.segs + 3) / 4, 3 * kCUs / p.rows)) : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes);
    return o;
  };
  const size_t rows = (size_t)p.rows, n = rows * (size_t)p.segs, h = rows * (size_t)p.splits;
  p.o_max = take(n * 4);
  p.o_min = take(n * 4);
  p.o_sum = take(n * 8);
  p.o_grp = take(n * 256);
  p.o_kept = take(n * 8);
  p.o_listed = take(rows * kLine * 4);
  p.o_hist = take(h * hist_bins_for(V) * 8);
  p.o_hist_n = take(h * hist_bins_for(V) * 4);
  p.o_z = take(h * 8);
  p.o_cut = take(hist ? rows * sizeof(RowCut) : 0);
  p.o_list = take(hist ? rows * kList * 8 : 0);
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
    const int64_t blocks = std::min<int64_t>((waves + 3) / 4, 1 << 20);
    k_sample_mass<T><<<(unsigned)blocks, 256, 0, s>>>(a, waves);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool k_on = a.k_rows != nullptr || (a.k > 0 && a.k < a.V);
  const bool p_on = a.p_rows != nullptr || (a.p > 0.0 && a.p < 1.0);
  const bool m_on = a.min_p_rows != nullptr || a.min_p > 0.0;
  const bool all_short = a.k_rows == nullptr && k_on && a.k <= kListK;   // LIST, whatever p
  if (a.V > kList && (k_on || p_on || m_on) && !all_short) {
    ScopedKernelTimer t(KK_SAMPLE_CUT, s);
    if (k_on || p_on) {
      const dim3 grid((unsigned)a.splits, (unsigned)rows);
      const bool few = a.V <= kFewBins;
      if (few) k_sample_hist<T, 2048><<<grid, kHistThreads, 0, s>>>(a);
      else k_sample_hist<T, 4096><<<grid, kHistThreads, 0, s>>>(a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if (few) k_sample_cut<2048><<<(unsigned)rows, kHistThreads, 0, s>>>(a);
      else k_sample_cut<4096><<<(unsigned)rows, kHistThreads, 0, s>>>(a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    k_sample_gather<T><<<dim3((unsigned)((a.segs + 3) / 4), (unsigned)rows), 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  ScopedKernelTimer t(KK_SAMPLE_PICK, s);
  if (k_on || p_on || m_on) k_sample_pick<T, true><<<(unsigned)rows, kPick, 0, s>>>(a);
  else k_sample_pick<T, false><<<(unsigned)rows, kPick, 0, s>>>(a);
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
  if ((uintptr_t)workspace % grpo::kAlign != 0)
    return fail(GRPO_ERR_WORKSPACE, "workspace is not 256-byte aligned");
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
    // 1 / T has to be finite: infinity times a difference of 0 is NaN
    a.T = o.temperature > 0.0 ? std::max(o.temperature, 1e-300) : 0.0;
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
    a.seg_kept = (uint64_t*)(ws + p.o_kept);
    a.listed = (int*)(ws + p.o_listed);
    a.hist = (uint64_t*)(ws + p.o_hist);
    a.hist_n = (uint32_t*)(ws + p.o_hist_n);
    a.z_part = (double*)(ws + p.o_z);
    a.cut = (grpo::RowCut*)(ws + p.o_cut);
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
