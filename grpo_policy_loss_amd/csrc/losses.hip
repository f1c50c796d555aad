// losses.hip -- losses over given log-probabilities and their gradients: the clipped policy
// loss with its KL term, and the preference loss over pairs.
//
// Both are sums over the tokens of padded sequences [B, L] with a mask, of values that need
// a sequence's own sums first where its ratio, its mean or its pair goes by them.  One pass
// over the tokens leaves float64 sums; what a sequence's sums decide is then worked out once
// for the sequence.  Two forms, by the length of the rows:
//   rows of at most 1024 tokens   a group of 1 to 64 lanes takes a whole sequence (or pair),
//   (8192 where they are many)    4 tokens a lane and load, so that its sums stay in a wave;
//                                 a block leaves one partial result of all its sequences
//   longer rows                   a block takes a segment of one sequence and leaves the
//                                 segment's sums; the finish joins a sequence's segments
// A second launch of one block finishes (none where one block held everything).  The backward
// goes token by token from what the forward kept of each sequence.
//
// Bound by memory where there are tokens enough: of 1021 rows of 16385 tokens with a sequence ratio and a
// KL term the forward reads 13 bytes a token in 42 us (5.2 TB/s), and the finish takes 9 us more; the
// backward moves 13 in 45 us (4.8 TB/s).  16384 pairs of 511 tokens, 5 bytes a token each way: 23 us
// (3.7 TB/s; float64 sums beside short rows) and 4, 17 us (4.9 TB/s).  Smaller ones are bound by launches:
// 8 rows of 20480 tokens 6.5, 4.4 and 4.8 us.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "api.hpp"
#include "elem.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

constexpr int kThreads = 256;
constexpr int kRowTokens = 1024;   // the longest row that a wave takes whole, or kManyTokens of
constexpr int kManyTokens = 8192;  // rows enough to fill the chip with waves
constexpr int kManyItems = 4096;
constexpr int kMaxBlocks = 1024;   // of the first form: 4 blocks on each of 256 CUs
constexpr int kMaxParts = 4096;    // segments of the second form, unless there are more rows
constexpr int kFinish = 1024;      // threads of the finish
// 2^24 tokens, us of the forward (clipped loss with an old and a reference policy | preference loss
// without one, 84 MB):
//                     8 tokens a lane   16          1 load ahead   4           2048 blocks
//   65536 rows of 256   60 | 29         54 | 25     68 | 42        83 | 36     59 | 25
//   32768 rows of 511   55 | 30         53 | 25     61 | 31        82 | 37     55 | 25
//   16384 rows of 1024  55 | 25         52 | 25     61 | 25        83 | 38     55 | 25
// (4 loads ahead leave two waves a SIMD, and 6 waves asked of the compiler spill: 114 | 43.)
constexpr int kAhead = 2;          // loads of each array that a lane has on their way
constexpr int kLaneTokens = 16;    // of a row that is shorter than 64 lanes' worth

typedef __attribute__((ext_vector_type(4), aligned(4))) float F4;
typedef __attribute__((ext_vector_type(4), aligned(1))) uint8_t U4;

// Four elements of a row of n for the lane whose turn is [c, c + 4): those, or the row's last four
// where they pass its end, so that no load is under a condition and several stay on their way.
// Rows of less than four read element by element, zeros behind them.
__device__ __forceinline__ F4 load4(const float* row, int c, int n) {
  if (n >= 4) return *(const F4*)(row + min(c, n - 4));
  F4 v = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < n) v[j] = row[c + j];
  return v;
}
__device__ __forceinline__ U4 load4(const uint8_t* row, int c, int n) {
  if (n >= 4) return *(const U4*)(row + min(c, n - 4));
  U4 v = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < n) v[j] = row[c + j];
  return v;
}
// Four gradients.  Non-temporal, so that the inputs stay in the caches rather: 1021 rows of 16385 tokens,
// both directions, 101 -> 91 us, 32768 of 511 111 -> 101, pairs 46.5 -> 42.7, 8 rows of 20480 16 either way.
// (Non-temporal loads in the forward take those of the backward out of the caches: 91 -> 93, 101 -> 112.)
__device__ __forceinline__ void store4(float* to, F4 v) { __builtin_nontemporal_store(v, (F4*)to); }
// The first of the four that is this lane's.
__device__ __forceinline__ int first4(int c, int n) { return n >= 4 ? c - min(c, n - 4) : 0; }

// Sums over the lanes of a group of `width` (a power of two up to 64).
template <typename T>
__device__ __forceinline__ T group_sum(T v, int width) {
  for (int o = width >> 1; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// e^x, e^x - 1 and e^x - 1 - x.  The last cancels near 0: there it is its series, and the others
// follow from it.  (x^2 (1 / 2 + x / 6 + ...): the first term left out is below 10^-10 of the sum.)
struct Exp {
  float e, em, excess;
};
__device__ __forceinline__ Exp exp_excess(float x) {
  float p = 1.f / 3628800;
  p = fmaf(p, x, 1.f / 362880);
  p = fmaf(p, x, 1.f / 40320);
  p = fmaf(p, x, 1.f / 5040);
  p = fmaf(p, x, 1.f / 720);
  p = fmaf(p, x, 1.f / 120);
  p = fmaf(p, x, 1.f / 24);
  p = fmaf(p, x, 1.f / 6);
  p = fmaf(p, x, 0.5f);
  p *= x * x;
  if (fabsf(x) < 0.5f) return {1.f + (x + p), x + p, p};
  const float e = expf(x);
  return {e, e - 1.f, (e - 1.f) - x};
}

// exp of a float64 value, to float32: the part of it that float32 loses comes in as a factor.
__device__ __forceinline__ float exp_wide(double x) {
  const float hi = (float)x;
  const float e = expf(hi);
  // (hi is infinite only where e is 0 or infinite)
  return fabsf(hi) < 200.f ? fmaf(e, (float)(x - (double)hi), e) : e;
}

// ---------------------------------------------------------------- clipped policy loss
struct ClipArgs {
  const float *lp, *old_lp, *ref_lp;
  const uint8_t* mask;
  const float* adv;
  float* weights;
  int64_t B;
  int32_t L;
  int32_t adv_per_token, seq_mean, kl;
  double log_high, log_low, log_dual;   // of the borders; infinite where there is none
  double high, low, dual, beta;         // the borders
};

// Which side of the borders a ratio of logarithm D is on, and what stands in for it: NaN is on
// neither.
struct Clipped {
  bool low, high;
};
template <typename T>
__device__ __forceinline__ Clipped clip_ratio(const ClipArgs& a, float adv, double D, T& s) {
  const bool above = adv >= 0.f && D > a.log_high, far = adv < 0.f && D > a.log_dual;
  const bool below = adv < 0.f && D < a.log_low;
  if (above) s = (T)a.high;
  if (below) s = (T)a.low;
  if (far) s = (T)a.dual;
  return {below, above || far};
}

// kl of one token, and its slope in lp (see grpo_opts for the estimators).
__device__ __forceinline__ float kl_term(int kind, float x, float lp) {
  const Exp v = exp_excess(x);
  // x e^x - (e^x - 1); near 0 as x (e^x - 1) - (e^x - 1 - x), which far below 0 would carry the rounding of x
  if (kind == GRPO_KL_FORWARD) return fabsf(x) < 0.5f ? fmaf(x, v.em, -v.excess) : fmaf(x, v.e, -v.em);
  if (kind == GRPO_KL_REVERSE_Q) return expf(lp) * v.excess;
  return v.excess;
}
__device__ __forceinline__ float kl_slope(int kind, float x, float lp) {
  if (kind == GRPO_KL_REVERSE_Q) return -x * expf(lp);
  const Exp v = exp_excess(x);
  return kind == GRPO_KL_FORWARD ? -x * v.e : -v.em;
}

// beta kl; where beta is 0 there is no such term, whatever kl is.
__device__ __forceinline__ double kl_weighed(const ClipArgs& a, double kl) {
  return a.beta != 0.0 ? a.beta * kl : 0.0;
}

struct ClipSums {
  double loss, d, kl, excess;
  int n, low, high, pad;
};

// Four tokens of a row of n that starts at token t0, and their part of the sums: loss is the policy
// term alone, and nothing where the ratio is the sequence's (SEQ).  A masked token counts as one with
// all logarithms 0 and no advantage, which adds nothing.  Policy terms, which may nearly cancel, go into
// float64 one by one.  The other terms are never negative: four of them first join in float32, which costs
// three roundings and no more.  Forward of 1021 rows of 16385 tokens | 16384 of 1024, us: the policy terms in two
// float64 sums in turn 53.5 | 47.2, in one 53.6 | 47.7, and all terms in float64 one by one 54.1 | 47.9.
template <bool SEQ>
struct ClipQuad {
  U4 m4;
  F4 lp4, old4, ref4, adv4;
  int first;

  __device__ __forceinline__ void load(const ClipArgs& a, int64_t t0, int c, int n) {
    first = first4(c, n);
    m4 = load4(a.mask + t0, c, n);
    lp4 = load4(a.lp + t0, c, n);
    if (a.old_lp != nullptr) old4 = load4(a.old_lp + t0, c, n);
    if (a.ref_lp != nullptr) ref4 = load4(a.ref_lp + t0, c, n);
    if (!SEQ && a.adv_per_token) adv4 = load4(a.adv + t0, c, n);
  }
  __device__ __forceinline__ void add(const ClipArgs& a, float adv_row, ClipSums& s) const {
    // quarters: four of float32's largest do not overflow
    float kl = 0.f, excess = 0.f;
    double loss[2] = {s.loss, 0.0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool m = m4[j] != 0 && j >= first;
      s.n += m;
      const float lp = m ? lp4[j] : 0.f;
      const double D = a.old_lp != nullptr ? (double)lp - (double)(m ? old4[j] : 0.f) : 0.0;
      if (SEQ) {
        s.d += D;
      } else {
        const float adv = m ? (a.adv_per_token ? adv4[j] : adv_row) : 0.f;
        const Exp v = exp_excess((float)D);
        float r = v.e;
        excess = fmaf(0.25f, v.excess, excess);
        const Clipped at = clip_ratio(a, adv, D, r);
        s.low += at.low;
        s.high += at.high;
        loss[j % 2] = fma(-(double)adv, (double)r, loss[j % 2]);
      }
      if (a.ref_lp != nullptr) kl = fmaf(0.25f, kl_term(a.kl, (m ? ref4[j] : 0.f) - lp, lp), kl);
    }
    s.kl = fma(4.0, (double)kl, s.kl);
    if (SEQ) return;
    s.loss = loss[0] + loss[1];
    s.excess = fma(4.0, (double)excess, s.excess);
  }
};

// All tokens of a row of n, `lanes` lanes apart, kAhead loads of each array ahead.
template <bool SEQ>
__device__ __forceinline__ void clip_row(const ClipArgs& a, int64_t t0, int n, int lane, int lanes,
                                         float adv, ClipSums& s) {
  for (int c = lane * 4; c < n; c += lanes * 4 * kAhead) {
    ClipQuad<SEQ> q[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) q[k].load(a, t0, c + k * lanes * 4, n);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) q[k].add(a, adv, s);
  }
}

// What the backward takes of a sequence: the factor of its terms, and its ratio's slope.
__device__ __forceinline__ void keep_sequence(const ClipArgs& a, int64_t b, float inv, float slope) {
  a.weights[2 * b] = inv;
  a.weights[2 * b + 1] = slope;
}

// What a sequence's own sums decide, in one lane for the sequence: the ratio's terms (SEQ; in
// float64, since a batch's advantages may nearly cancel), and what the backward takes of it.  Gives
// the factor of the sequence's loss.
template <bool SEQ>
__device__ __forceinline__ double clip_sequence(const ClipArgs& a, int64_t b, float adv, int n,
                                                double d, bool writes, ClipSums& s) {
  const double inv = a.seq_mean && n > 0 ? 1.0 / n : 1.0;
  float slope = 0.f;
  if (SEQ) {
    const double D = n > 0 ? d / n : 0.0;
    const double r = exp(D);
    double used = r;
    const Clipped at = clip_ratio(a, adv, D, used);
    if (!at.low && !at.high) slope = (float)(-adv * r);
    if (writes && n > 0) {
      s.low += at.low ? n : 0;
      s.high += at.high ? n : 0;
      s.excess += (expm1(D) - D) * n;
      s.loss -= adv * used * n;
    }
  }
  if (writes) keep_sequence(a, b, (float)inv, slope);
  return inv;
}

// The sums of all threads of the block, in thread 0.
template <int THREADS>
__device__ __forceinline__ void clip_block_sum(ClipSums& s) {
  __shared__ ClipSums waves[THREADS / 64];
  s.loss = group_sum(s.loss, 64);
  s.d = group_sum(s.d, 64);
  s.kl = group_sum(s.kl, 64);
  s.excess = group_sum(s.excess, 64);
  s.n = group_sum(s.n, 64);
  s.low = group_sum(s.low, 64);
  s.high = group_sum(s.high, 64);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / 64; ++w) {
      s.loss += waves[w].loss;
      s.d += waves[w].d;
      s.kl += waves[w].kl;
      s.excess += waves[w].excess;
      s.n += waves[w].n;
      s.low += waves[w].low;
      s.high += waves[w].high;
    }
}

// The results from the sums of everything (one thread).
__device__ __forceinline__ void clip_result(const ClipArgs& a, const ClipSums& s, float* loss,
                                            float* stats) {
  const double n = s.n > 0 ? s.n : 1, den = a.seq_mean ? (double)a.B : n;
  loss[0] = (float)(s.loss / den);
  a.weights[2 * a.B] = (float)(1.0 / den);
  stats[0] = (float)(s.kl / n);
  stats[1] = (float)(s.low / n);
  stats[2] = (float)(s.high / n);
  stats[3] = (float)(s.excess / n);
}

// Rows of at most kRowTokens tokens, a group of `width` lanes each.
template <bool SEQ>
__global__ void __launch_bounds__(kThreads)
    k_clip_rows(ClipArgs a, int width, ClipSums* __restrict__ parts, float* __restrict__ loss,
                float* __restrict__ stats) {
  const int lane = threadIdx.x & (width - 1);
  const int64_t groups = (int64_t)gridDim.x * (kThreads / width);
  // (adjacent lanes, adjacent sequences: by one lane in the loop below 48.0 in the place of 47.2 us)
  if (!SEQ && !a.seq_mean)
    for (int64_t b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += (int64_t)gridDim.x * kThreads)
      keep_sequence(a, b, 1.f, 0.f);
  ClipSums s = {};
  for (int64_t b = (int64_t)blockIdx.x * (kThreads / width) + threadIdx.x / width; b < a.B; b += groups) {
    const float adv = a.adv_per_token ? 0.f : a.adv[b];
    ClipSums row = {};
    clip_row<SEQ>(a, b * a.L, a.L, lane, width, adv, row);
    const int n = row.n;
    double inv = 1.0;
    if (SEQ || a.seq_mean) {
      const int all = group_sum(n, width);
      const double d = SEQ ? group_sum(row.d, width) : 0.0;
      inv = clip_sequence<SEQ>(a, b, adv, all, d, lane == 0, row);
    }
    s.loss += (row.loss + kl_weighed(a, row.kl)) * inv;
    s.kl += row.kl;
    s.excess += row.excess;
    s.n += n;
    s.low += row.low;
    s.high += row.high;
  }
  clip_block_sum<kThreads>(s);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) clip_result(a, s, loss, stats);
  else parts[blockIdx.x] = s;
}

// Longer rows: block `seg` of `segs` of row b, `span` tokens.
template <bool SEQ>
__global__ void __launch_bounds__(kThreads)
    k_clip_segments(ClipArgs a, int segs, int span, ClipSums* __restrict__ parts) {
  const int64_t b = blockIdx.x / (unsigned)segs;
  const int seg = (int)(blockIdx.x - b * segs);
  const float adv = a.adv_per_token ? 0.f : a.adv[b];
  const int64_t from = (int64_t)seg * span;
  const int n = (int)min<int64_t>(span, a.L - from);
  ClipSums s = {};
  clip_row<SEQ>(a, b * a.L + from, n, threadIdx.x, kThreads, adv, s);
  clip_block_sum<kThreads>(s);
  if (threadIdx.x != 0) return;
  parts[blockIdx.x] = s;
  if (!SEQ && !a.seq_mean && seg == 0) keep_sequence(a, b, 1.f, 0.f);
}

// The finish: of blocks' sums (segs 0), or of rows' segments, `width` lanes for a row.
template <bool SEQ>
__global__ void __launch_bounds__(kFinish)
    k_clip_finish(ClipArgs a, const ClipSums* __restrict__ parts, int count, int segs, int width,
                  float* __restrict__ loss, float* __restrict__ stats) {
  ClipSums s = {};
  if (segs == 0) {
    for (int i = threadIdx.x; i < count; i += kFinish) {
      const ClipSums p = parts[i];
      s.loss += p.loss;
      s.kl += p.kl;
      s.excess += p.excess;
      s.n += p.n;
      s.low += p.low;
      s.high += p.high;
    }
  } else {
    const int lane = threadIdx.x & (width - 1);
    for (int64_t b = threadIdx.x / width; b < a.B; b += kFinish / width) {
      ClipSums row = {};
#pragma unroll 4
      for (int i = lane; i < segs; i += width) {
        const ClipSums p = parts[b * segs + i];
        row.loss += p.loss;
        row.d += p.d;
        row.kl += p.kl;
        row.excess += p.excess;
        row.n += p.n;
        row.low += p.low;
        row.high += p.high;
      }
      const int n = row.n;
      double inv = 1.0;
      if (SEQ || a.seq_mean) {
        const float adv = a.adv_per_token ? 0.f : a.adv[b];
        const int all = group_sum(n, width);
        const double d = SEQ ? group_sum(row.d, width) : 0.0;
        inv = clip_sequence<SEQ>(a, b, adv, all, d, lane == 0, row);
      }
      s.loss += (row.loss + kl_weighed(a, row.kl)) * inv;
      s.kl += row.kl;
      s.excess += row.excess;
      s.n += n;
      s.low += row.low;
      s.high += row.high;
    }
  }
  clip_block_sum<kFinish>(s);
  if (threadIdx.x == 0) clip_result(a, s, loss, stats);
}

// t / L for 0 <= t < 2^31: with 2^(s-1) < L <= 2^s and mul = ceil(2^(31+s) / L), t mul / 2^(31+s)
// is less than 1 / L above t / L.
struct Divide {
  uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t divide(uint32_t t, Divide by) {
  return (uint32_t)((uint64_t)t * by.mul >> by.shift);
}

// Four tokens a lane, whatever rows they are in.
template <bool SEQ>
__global__ void __launch_bounds__(kThreads)
    k_clip_bwd(ClipArgs a, Divide by, int64_t N, const float* __restrict__ grad_loss,
               float* __restrict__ grad_lp) {
  const int64_t t0 = (int64_t)blockIdx.x * (kThreads * 4);
  const int n = (int)min<int64_t>(kThreads * 4, N - t0);
  int c = threadIdx.x * 4;
  if (c >= n) return;
  c -= first4(c, n);     // where they pass the end, two lanes form the same gradients
  float g = a.weights[2 * a.B];
  if (grad_loss != nullptr) g *= *grad_loss;
  const U4 m4 = load4(a.mask + t0, c, n);
  F4 lp4 = {}, old4 = {}, ref4 = {}, adv4 = {};
  lp4 = load4(a.lp + t0, c, n);
  if (!SEQ && a.old_lp != nullptr) old4 = load4(a.old_lp + t0, c, n);
  if (a.ref_lp != nullptr) ref4 = load4(a.ref_lp + t0, c, n);
  if (a.adv_per_token) adv4 = load4(a.adv + t0, c, n);
  F4 out;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool m = m4[j] != 0;
    const uint32_t b = divide((uint32_t)min<int64_t>(t0 + c + j, N - 1), by);
    const float lp = m ? lp4[j] : 0.f;
    float w = g, slope;
    if (a.seq_mean) w *= a.weights[2 * (int64_t)b];
    if (SEQ) {
      slope = a.weights[2 * (int64_t)b + 1];
    } else {
      const float adv = a.adv_per_token ? adv4[j] : a.adv[b];
      const double D = a.old_lp != nullptr ? (double)lp - (double)(m ? old4[j] : 0.f) : 0.0;
      float r = exp_excess((float)D).e;
      const Clipped at = clip_ratio(a, adv, D, r);
      slope = at.low || at.high ? 0.f : -adv * r;
    }
    if (a.ref_lp != nullptr) slope = fmaf((float)a.beta, kl_slope(a.kl, (m ? ref4[j] : 0.f) - lp, lp), slope);
    out[j] = m ? w * slope : 0.f;
  }
  if (c + 4 <= n) {
    store4(grad_lp + t0 + c, out);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < n) grad_lp[t0 + c + j] = out[j];
  }
}

// ---------------------------------------------------------------- preference loss
struct PrefArgs {
  const float *lp, *ref_lp;
  const uint8_t* mask;
  float *rewards, *weights;
  int64_t P;
  int32_t L;
  int32_t kind, length_mean;
  double beta, smoothing, margin, nll;
};

struct PrefSums {
  double d, lp;
  int n, pad;
};

struct PrefQuad {
  U4 m4;
  F4 lp4, ref4;
  int first;

  __device__ __forceinline__ void load(const PrefArgs& a, int64_t t0, int c, int n) {
    first = first4(c, n);
    m4 = load4(a.mask + t0, c, n);
    lp4 = load4(a.lp + t0, c, n);
    if (a.ref_lp != nullptr) ref4 = load4(a.ref_lp + t0, c, n);
  }
  __device__ __forceinline__ void add(const PrefArgs& a, PrefSums& s) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool m = m4[j] != 0 && j >= first;
      const double lp = m ? (double)lp4[j] : 0.0;
      s.n += m;
      s.lp += lp;
      if (a.ref_lp != nullptr) s.d += lp - (m ? (double)ref4[j] : 0.0);
    }
  }
};

// All tokens of `ROWS` rows of n that lie `apart` tokens apart.
template <int ROWS>
__device__ __forceinline__ void pref_row(const PrefArgs& a, int64_t t0, int64_t apart, int n, int lane,
                                         int lanes, PrefSums (&s)[ROWS]) {
  for (int c = lane * 4; c < n; c += lanes * 4 * kAhead) {
    PrefQuad q[ROWS][kAhead];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int k = 0; k < kAhead; ++k) q[r][k].load(a, t0 + r * apart, c + k * lanes * 4, n);
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int k = 0; k < kAhead; ++k) q[r][k].add(a, s[r]);
  }
}

// log(1 + e^x) and sigmoid(x), of a float64 x.
__device__ __forceinline__ void softplus(double x, double& value, double& slope) {
  const float e = exp_wide(-fabs(x));          // NaN stays
  const float l = log1pf(e), q = 1.f / (1.f + e);
  value = fmax(x, 0.0) + (double)l;
  slope = (double)(x >= 0.0 ? q : e * q);
}

// The loss of pair p from its sequences' sums (c chosen, r rejected), and what the backward and
// the user take of it.
__device__ __forceinline__ double pref_pair(const PrefArgs& a, int64_t p, PrefSums c, PrefSums r) {
  const double nc = c.n > 0 ? c.n : 1, nr = r.n > 0 ? r.n : 1;
  double sc = a.ref_lp != nullptr ? c.d : c.lp, sr = a.ref_lp != nullptr ? r.d : r.lp;
  if (a.length_mean) sc /= nc, sr /= nr;
  const double h = sc - sr, x = a.beta * h - a.margin;
  double loss, slope;   // in h
  if (a.kind == GRPO_PREF_SIGMOID) {
    // -(1 - e) log sigmoid(x) - e log sigmoid(-x), with softplus(x) = softplus(-x) + x
    double lo, so, hi, si;
    softplus(-x, lo, so);
    softplus(x, hi, si);
    loss = a.smoothing != 0.0 ? (1.0 - a.smoothing) * lo + a.smoothing * hi : lo;
    slope = a.beta * (a.smoothing != 0.0 ? a.smoothing * si - (1.0 - a.smoothing) * so : -so);
  } else if (a.kind == GRPO_PREF_HINGE) {
    loss = x > 1.0 ? 0.0 : 1.0 - x;
    slope = x >= 1.0 ? 0.0 : -a.beta;
    if (x != x) slope = x;
  } else {
    const double off = h - a.margin - 0.5 / a.beta;
    loss = off * off;
    slope = 2.0 * off;
  }
  const double share = slope / (double)a.P;
  double wc = a.length_mean ? share / nc : share;
  const double wr = a.length_mean ? share / nr : share;
  if (a.nll != 0.0) {
    loss -= a.nll * (c.lp / nc);
    wc -= a.nll / (nc * (double)a.P);
  }
  a.rewards[2 * p] = (float)(a.beta * sc);
  a.rewards[2 * p + 1] = (float)(a.beta * sr);
  a.weights[2 * p] = (float)wc;
  a.weights[2 * p + 1] = (float)-wr;
  return loss;
}

__device__ __forceinline__ PrefSums pref_group_sum(PrefSums s, int width, bool with_lp, bool with_d) {
  if (with_d) s.d = group_sum(s.d, width);
  if (with_lp) s.lp = group_sum(s.lp, width);
  s.n = group_sum(s.n, width);
  return s;
}

template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double waves[THREADS / 64];
  v = group_sum(v, 64);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / 64; ++w) v += waves[w];
  return v;
}

__global__ void __launch_bounds__(kThreads)
    k_pref_rows(PrefArgs a, int width, double* __restrict__ parts, float* __restrict__ loss) {
  const int lane = threadIdx.x & (width - 1);
  const int64_t groups = (int64_t)gridDim.x * (kThreads / width);
  const bool with_d = a.ref_lp != nullptr, with_lp = !with_d || a.nll != 0.0;
  double s = 0.0;
  for (int64_t p = (int64_t)blockIdx.x * (kThreads / width) + threadIdx.x / width; p < a.P; p += groups) {
    PrefSums two[2] = {};
    pref_row<2>(a, 2 * p * a.L, a.L, a.L, lane, width, two);
    const PrefSums chosen = pref_group_sum(two[0], width, with_lp, with_d);
    const PrefSums rejected = pref_group_sum(two[1], width, with_lp, with_d);
    if (lane == 0) s += pref_pair(a, p, chosen, rejected);
  }
  s = block_sum<kThreads>(s);
  if (threadIdx.x != 0) return;
  if (gridDim.x == 1) loss[0] = (float)(s / (double)a.P);
  else parts[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads)
    k_pref_segments(PrefArgs a, int segs, int span, PrefSums* __restrict__ parts) {
  const int64_t b = blockIdx.x / (unsigned)segs;
  const int64_t from = (int64_t)(blockIdx.x - b * segs) * span;
  const int n = (int)min<int64_t>(span, a.L - from);
  PrefSums one[1] = {};
  pref_row<1>(a, b * a.L + from, 0, n, threadIdx.x, kThreads, one);
  __shared__ PrefSums waves[kThreads / 64];
  PrefSums s = pref_group_sum(one[0], 64, true, true);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 64; ++w) {
    s.d += waves[w].d;
    s.lp += waves[w].lp;
    s.n += waves[w].n;
  }
  parts[blockIdx.x] = s;
}

// The finish: of blocks' losses (segs 0), or of pairs' segments, `width` lanes for a pair.
__global__ void __launch_bounds__(kFinish)
    k_pref_finish(PrefArgs a, const void* __restrict__ parts, int count, int segs, int width,
                  float* __restrict__ loss) {
  double s = 0.0;
  if (segs == 0) {
    for (int i = threadIdx.x; i < count; i += kFinish) s += ((const double*)parts)[i];
  } else {
    const int lane = threadIdx.x & (width - 1);
    const PrefSums* rows = (const PrefSums*)parts;
    for (int64_t p = threadIdx.x / width; p < a.P; p += kFinish / width) {
      PrefSums two[2] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll 4
        for (int i = lane; i < segs; i += width) {
          const PrefSums q = rows[(2 * p + k) * segs + i];
          two[k].d += q.d;
          two[k].lp += q.lp;
          two[k].n += q.n;
        }
        two[k] = pref_group_sum(two[k], width, true, true);
      }
      if (lane == 0) s += pref_pair(a, p, two[0], two[1]);
    }
  }
  s = block_sum<kFinish>(s);
  if (threadIdx.x == 0) loss[0] = (float)(s / (double)a.P);
}

__global__ void __launch_bounds__(kThreads)
    k_pref_bwd(const uint8_t* __restrict__ mask, const float* __restrict__ weights,
               const float* __restrict__ grad_loss, Divide by, int64_t N,
               float* __restrict__ grad_lp) {
  const int64_t t0 = (int64_t)blockIdx.x * (kThreads * 4);
  const int n = (int)min<int64_t>(kThreads * 4, N - t0);
  int c = threadIdx.x * 4;
  if (c >= n) return;
  c -= first4(c, n);
  const float g = grad_loss != nullptr ? *grad_loss : 1.f;
  const U4 m4 = load4(mask + t0, c, n);
  F4 out;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = divide((uint32_t)min<int64_t>(t0 + c + j, N - 1), by);
    out[j] = m4[j] != 0 ? g * weights[b] : 0.f;
  }
  if (c + 4 <= n) {
    store4(grad_lp + t0 + c, out);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < n) grad_lp[t0 + c + j] = out[j];
  }
}

// ---------------------------------------------------------------- plans
inline int pow2_at_least(int64_t x, int most) {
  int p = 1;
  while (p < x && p < most) p *= 2;
  return p;
}

// How `items` (sequences, or pairs of two) of `rows` rows of L tokens are split.
struct Split {
  int width;         // lanes of an item, where waves take them whole
  int segs, span;    // or blocks of a row and their tokens
  int blocks;        // of the first launch
  int parts;         // that it leaves (0: it finishes)
  int finish_width;  // lanes of an item in the finish
};

Split split_rows(int64_t items, int64_t rows, int64_t L) {
  Split p{};
  if (L <= kRowTokens || (items >= kManyItems && L <= kManyTokens)) {
    p.width = pow2_at_least((L + kLaneTokens - 1) / kLaneTokens, 64);
    const int64_t per = kThreads / p.width;
    p.blocks = (int)std::min<int64_t>((items + per - 1) / per, kMaxBlocks);
    p.parts = p.blocks == 1 ? 0 : p.blocks;
    p.finish_width = 1;
    return p;
  }
  int64_t span = kRowTokens;
  while (span < L && rows * ((L + span - 1) / span) > kMaxParts) span *= 2;
  p.segs = (int)((L + span - 1) / span);
  // even segments, of whole loads
  p.span = (int)(((L + p.segs - 1) / p.segs + 3) / 4 * 4);
  p.segs = (int)((L + p.span - 1) / p.span);
  p.blocks = p.parts = (int)(rows * p.segs);
  // lanes for all of a row's segments, but no more than let every row have its turn at once (forward
  // with a sequence ratio: 200 rows of 20000 tokens 29 -> 21 us, 1021 of 16385 37 -> 35)
  p.finish_width = pow2_at_least(p.segs, 64);
  while (p.finish_width > 1 && items * p.finish_width > kFinish) p.finish_width /= 2;
  return p;
}

Divide divider(int64_t L) {
  uint32_t s = 0;
  while (((int64_t)1 << s) < L) ++s;
  const unsigned __int128 num = (unsigned __int128)1 << (31 + s);
  return {(uint32_t)((num + (uint64_t)L - 1) / (uint64_t)L), 31 + s};
}

// rows * L tokens: positive, and no more than fit int32.
int check_rows(int64_t rows, int64_t L, int64_t per) {
  if (rows <= 0 || L <= 0) return fail(GRPO_ERR_INVALID_ARG, "sizes must be positive (%lld, L=%lld)",
                                       (long long)rows, (long long)L);
  if (rows > INT32_MAX / per || L > INT32_MAX / (rows * per))
    return fail(GRPO_ERR_UNSUPPORTED, "more tokens than fit int32");
  return GRPO_OK;
}

int check_workspace(const void* ws, size_t got, size_t need) {
  if (ws == nullptr || got < need)
    return fail(GRPO_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, ws == nullptr ? (size_t)0 : got);
  if ((uintptr_t)ws % kAlign != 0) return fail(GRPO_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  return GRPO_OK;
}

int clip_args(const float* lp, const float* old_lp, const float* ref_lp, const uint8_t* mask,
              const float* adv, const float* weights, int64_t B, int64_t L,
              const grpo_clip_opts* opts, ClipArgs* a) {
  const grpo_clip_opts none{};
  const grpo_clip_opts& o = opts != nullptr ? *opts : none;
  GRPO_CHECK_PTR(lp);
  GRPO_CHECK_PTR(mask);
  GRPO_CHECK_PTR(adv);
  GRPO_CHECK_PTR(weights);
  const int st = check_rows(B, L, 1);
  if (st != GRPO_OK) return st;
  if (!(o.clip_low >= 0.0 && o.clip_low <= FLT_MAX && o.clip_high >= 0.0 && o.clip_high <= FLT_MAX))
    return fail(GRPO_ERR_INVALID_ARG, "clip_low and clip_high must be finite in float32 and >= 0 (%g, %g)", o.clip_low,
                o.clip_high);
  if (!(o.clip_dual == 0.0 || (o.clip_dual > 1.0 && o.clip_dual <= FLT_MAX)))
    return fail(GRPO_ERR_INVALID_ARG, "clip_dual must be 0 or above 1 and finite in float32 (%g)", o.clip_dual);
  if (!(fabs(o.beta) <= FLT_MAX)) return fail(GRPO_ERR_INVALID_ARG, "beta must be finite in float32");
  if (o.beta != 0.0 && ref_lp == nullptr) return fail(GRPO_ERR_INVALID_ARG, "beta %g needs ref_lp", o.beta);
  if (o.ratio != GRPO_RATIO_TOKEN && o.ratio != GRPO_RATIO_SEQUENCE)
    return fail(GRPO_ERR_INVALID_ARG, "ratio %d is not 0 or 1", (int)o.ratio);
  if (o.kl_estimator < GRPO_KL_REVERSE || o.kl_estimator > GRPO_KL_REVERSE_Q)
    return fail(GRPO_ERR_INVALID_ARG, "kl_estimator %d is not 0, 1 or 2", (int)o.kl_estimator);
  if (o.aggregation != GRPO_AGG_TOKEN_MEAN && o.aggregation != GRPO_AGG_SEQUENCE_MEAN)
    return fail(GRPO_ERR_INVALID_ARG, "aggregation %d is not 0 or 1", (int)o.aggregation);
  if (o.adv_per_token != 0 && o.adv_per_token != 1)
    return fail(GRPO_ERR_INVALID_ARG, "adv_per_token %d is not 0 or 1", (int)o.adv_per_token);
  if (o.adv_per_token && o.ratio == GRPO_RATIO_SEQUENCE)
    return fail(GRPO_ERR_INVALID_ARG, "a ratio for each sequence takes one advantage for each sequence");
  *a = ClipArgs{lp, old_lp, ref_lp, mask, adv, const_cast<float*>(weights), B, (int32_t)L,
                o.adv_per_token, o.aggregation == GRPO_AGG_SEQUENCE_MEAN, o.kl_estimator,
                HUGE_VAL, -HUGE_VAL, HUGE_VAL, 0.0, 0.0, 0.0, o.beta};
  if (o.clip_high > 0.0) a->log_high = log1p(o.clip_high), a->high = 1.0 + o.clip_high;
  // at 1 and beyond nothing is clipped from below: a ratio is not negative
  if (o.clip_low > 0.0 && o.clip_low < 1.0) a->log_low = log1p(-o.clip_low), a->low = 1.0 - o.clip_low;
  if (o.clip_dual > 0.0) a->log_dual = log(o.clip_dual), a->dual = o.clip_dual;
  return GRPO_OK;
}

template <bool SEQ>
int clip_forward(const ClipArgs& a, float* loss, float* stats, void* ws, hipStream_t s) {
  const Split p = split_rows(a.B, a.B, a.L);
  ClipSums* parts = (ClipSums*)ws;
  {
    ScopedKernelTimer timer(KK_CLIP_FWD, s);
    if (p.segs == 0) k_clip_rows<SEQ><<<(unsigned)p.blocks, kThreads, 0, s>>>(a, p.width, parts, loss, stats);
    else k_clip_segments<SEQ><<<(unsigned)p.blocks, kThreads, 0, s>>>(a, p.segs, p.span, parts);
    GRPO_HIP(hipGetLastError());
  }
  if (p.parts == 0) return GRPO_OK;
  ScopedKernelTimer timer(KK_LOSS_FINISH, s);
  k_clip_finish<SEQ><<<1, kFinish, 0, s>>>(a, parts, p.parts, p.segs, p.finish_width, loss, stats);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

}  // namespace
}  // namespace grpo

using grpo::fail;

extern "C" {

size_t grpo_clip_loss_workspace_bytes(int64_t B, int64_t L) {
  grpo::clear_error();
  if (grpo::check_rows(B, L, 1) != GRPO_OK) return 0;
  return grpo::align_up((size_t)std::max(1, grpo::split_rows(B, B, L).parts) * sizeof(grpo::ClipSums));
}

int grpo_clip_loss_fwd(const float* lp, const float* old_lp, const float* ref_lp,
                       const uint8_t* mask, const float* adv, int64_t B, int64_t L,
                       const grpo_clip_opts* opts, float* loss, float* stats, float* weights,
                       void* workspace, size_t workspace_bytes, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(loss);
  GRPO_CHECK_PTR(stats);
  grpo::ClipArgs a;
  int st = grpo::clip_args(lp, old_lp, ref_lp, mask, adv, weights, B, L, opts, &a);
  if (st != GRPO_OK) return st;
  const size_t need = grpo_clip_loss_workspace_bytes(B, L);
  st = grpo::check_workspace(workspace, workspace_bytes, need);
  if (st != GRPO_OK) return st;
  const size_t n = (size_t)(B * L);
  if (!grpo::apart({{loss, 4}, {stats, 16}, {weights, (2 * (size_t)B + 1) * 4}, {workspace, need}},
                   {{lp, 4 * n}, {old_lp, 4 * n}, {ref_lp, 4 * n}, {mask, n}, {adv, 4 * (a.adv_per_token ? n : (size_t)B)}}))
    return fail(GRPO_ERR_INVALID_ARG, "loss, stats, weights or workspace overlaps an input or another of them");
  const bool seq = opts != nullptr && opts->ratio == GRPO_RATIO_SEQUENCE;
  return seq ? grpo::clip_forward<true>(a, loss, stats, workspace, (hipStream_t)stream)
             : grpo::clip_forward<false>(a, loss, stats, workspace, (hipStream_t)stream);
}

int grpo_clip_loss_bwd(const float* lp, const float* old_lp, const float* ref_lp,
                       const uint8_t* mask, const float* adv, const float* weights,
                       const float* grad_loss, int64_t B, int64_t L, const grpo_clip_opts* opts,
                       float* grad_lp, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(grad_lp);
  grpo::ClipArgs a;
  const int st = grpo::clip_args(lp, old_lp, ref_lp, mask, adv, weights, B, L, opts, &a);
  if (st != GRPO_OK) return st;
  const size_t n = (size_t)(B * L);
  if (!grpo::apart({{grad_lp, 4 * n}},
                   {{lp, 4 * n}, {old_lp, 4 * n}, {ref_lp, 4 * n}, {mask, n}, {adv, 4 * (a.adv_per_token ? n : (size_t)B)},
                    {weights, (2 * (size_t)B + 1) * 4}, {grad_loss, 4}}))
    return fail(GRPO_ERR_INVALID_ARG, "grad_lp overlaps an input");
  hipStream_t s = (hipStream_t)stream;
  grpo::ScopedKernelTimer timer(grpo::KK_CLIP_BWD, s);
  const int64_t N = B * L;
  const unsigned blocks = (unsigned)((N + grpo::kThreads * 4 - 1) / (grpo::kThreads * 4));
  const grpo::Divide by = grpo::divider(L);
  if (a.beta == 0.0) a.ref_lp = nullptr;
  if (opts != nullptr && opts->ratio == GRPO_RATIO_SEQUENCE)
    grpo::k_clip_bwd<true><<<blocks, grpo::kThreads, 0, s>>>(a, by, N, grad_loss, grad_lp);
  else
    grpo::k_clip_bwd<false><<<blocks, grpo::kThreads, 0, s>>>(a, by, N, grad_loss, grad_lp);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

size_t grpo_pref_loss_workspace_bytes(int64_t P, int64_t L) {
  grpo::clear_error();
  if (grpo::check_rows(P, L, 2) != GRPO_OK) return 0;
  return grpo::align_up((size_t)std::max(1, grpo::split_rows(P, 2 * P, L).parts) * sizeof(grpo::PrefSums));
}

int grpo_pref_loss_fwd(const float* lp, const float* ref_lp, const uint8_t* mask, int64_t P,
                       int64_t L, const grpo_pref_opts* opts, float* loss, float* rewards,
                       float* weights, void* workspace, size_t workspace_bytes, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(lp);
  GRPO_CHECK_PTR(mask);
  GRPO_CHECK_PTR(opts);
  GRPO_CHECK_PTR(loss);
  GRPO_CHECK_PTR(rewards);
  GRPO_CHECK_PTR(weights);
  int st = grpo::check_rows(P, L, 2);
  if (st != GRPO_OK) return st;
  const grpo_pref_opts& o = *opts;
  if (!(o.beta > 0.0 && o.beta <= FLT_MAX)) return fail(GRPO_ERR_INVALID_ARG, "beta must be finite and > 0 (%g)", o.beta);
  if (!(fabs(o.margin) <= FLT_MAX && o.nll_weight >= 0.0 && o.nll_weight <= FLT_MAX))
    return fail(GRPO_ERR_INVALID_ARG, "margin and nll_weight must be finite, and nll_weight >= 0 (%g, %g)", o.margin,
                o.nll_weight);
  if (o.kind != GRPO_PREF_SIGMOID && o.kind != GRPO_PREF_HINGE && o.kind != GRPO_PREF_SQUARE)
    return fail(GRPO_ERR_INVALID_ARG, "kind %d is not 0, 1 or 2", (int)o.kind);
  if (!(o.label_smoothing >= 0.0 && o.label_smoothing < 1.0) ||
      (o.label_smoothing != 0.0 && o.kind != GRPO_PREF_SIGMOID))
    return fail(GRPO_ERR_INVALID_ARG, "label_smoothing must be in [0, 1), and 0 but for GRPO_PREF_SIGMOID (%g)",
                o.label_smoothing);
  if (o.length_mean != 0 && o.length_mean != 1)
    return fail(GRPO_ERR_INVALID_ARG, "length_mean %d is not 0 or 1", (int)o.length_mean);
  const size_t need = grpo_pref_loss_workspace_bytes(P, L), n = (size_t)(2 * P * L), rows = (size_t)(2 * P);
  st = grpo::check_workspace(workspace, workspace_bytes, need);
  if (st != GRPO_OK) return st;
  if (!grpo::apart({{loss, 4}, {rewards, 4 * rows}, {weights, 4 * rows}, {workspace, need}},
                   {{lp, 4 * n}, {ref_lp, 4 * n}, {mask, n}}))
    return fail(GRPO_ERR_INVALID_ARG, "loss, rewards, weights or workspace overlaps an input or another of them");
  const grpo::PrefArgs a{lp, ref_lp, mask, rewards, weights, P, (int32_t)L, o.kind, o.length_mean, o.beta,
                         o.label_smoothing, o.margin, o.nll_weight};
  const grpo::Split p = grpo::split_rows(P, 2 * P, L);
  hipStream_t s = (hipStream_t)stream;
  {
    grpo::ScopedKernelTimer timer(grpo::KK_PREF_FWD, s);
    if (p.segs == 0)
      grpo::k_pref_rows<<<(unsigned)p.blocks, grpo::kThreads, 0, s>>>(a, p.width, (double*)workspace, loss);
    else
      grpo::k_pref_segments<<<(unsigned)p.blocks, grpo::kThreads, 0, s>>>(a, p.segs, p.span,
                                                                         (grpo::PrefSums*)workspace);
    GRPO_HIP(hipGetLastError());
  }
  if (p.parts == 0) return GRPO_OK;
  grpo::ScopedKernelTimer timer(grpo::KK_LOSS_FINISH, s);
  grpo::k_pref_finish<<<1, grpo::kFinish, 0, s>>>(a, workspace, p.parts, p.segs, p.finish_width, loss);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

int grpo_pref_loss_bwd(const uint8_t* mask, const float* weights, const float* grad_loss,
                       int64_t P, int64_t L, float* grad_lp, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(mask);
  GRPO_CHECK_PTR(weights);
  GRPO_CHECK_PTR(grad_lp);
  const int st = grpo::check_rows(P, L, 2);
  if (st != GRPO_OK) return st;
  const int64_t N = 2 * P * L;
  if (!grpo::apart({{grad_lp, 4 * (size_t)N}}, {{mask, (size_t)N}, {weights, 8 * (size_t)P}, {grad_loss, 4}}))
    return fail(GRPO_ERR_INVALID_ARG, "grad_lp overlaps an input");
  hipStream_t s = (hipStream_t)stream;
  grpo::ScopedKernelTimer timer(grpo::KK_PREF_BWD, s);
  const unsigned blocks = (unsigned)((N + grpo::kThreads * 4 - 1) / (grpo::kThreads * 4));
  grpo::k_pref_bwd<<<blocks, grpo::kThreads, 0, s>>>(mask, weights, grad_loss, grpo::divider(L), N, grad_lp);
  GRPO_HIP(hipGetLastError());
  return GRPO_OK;
}

}  // extern "C"
