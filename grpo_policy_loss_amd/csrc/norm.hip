// norm.hip -- layer norm and RMS norm of rows, forward and backward.
//
// A row x of n elements, mu = mean(x) (0 for RMS), r = 1 / sqrt(mean((x - mu)^2) + eps),
// xh = (x - mu) r:
//   y  = xh w + b
//   dx = r (g - mean(g) - xh mean(g xh)),  g = dy w        (no mean(g) term for RMS)
//   dw += sum over rows of dy xh,  db += sum over rows of dy
// All of it is bound by memory: the forward reads x once and writes y once, the backward
// reads dy and x once and writes dx once.  A row therefore stays in registers between its
// sums and its result: LPR lanes hold a row as NV vectors of 16 bytes each.  Measured in bf16:
// forward of 32768 x 1536 39 us (5.2 TB/s), backward of 32768 x 4096 with mean and bias 148 us
// (5.4 TB/s); a copy of that size reaches 4.7 to 5.1 TB/s on the same card.
#include <math.h>

#include <algorithm>

#include "api.hpp"
#include "elem.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

constexpr int kCUs = 256;

template <int LPR> constexpr int kThreads = LPR > 256 ? LPR : 256;
// The backward takes two rows of 256 lanes at a time: a block then leaves one partial row of dw
// for twice the rows.
template <int LPR> constexpr int kThreadsBwd = LPR >= 256 && LPR <= 512 ? 512 : kThreads<LPR>;

// Sums of a and b over the LPR lanes of a row, in every lane.  LPR > 64: the waves' sums meet
// in LDS.  `phase` alternates between two LDS buffers, so one barrier
// per call is enough: a buffer is written again only behind the next call's barrier, which
// every wave reaches after it has read this one.
template <int LPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*lds)[2][16], int phase) {
#pragma unroll
  for (int o = (LPR < 64 ? LPR : 64) / 2; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int w = threadIdx.x >> 6, w0 = threadIdx.x / LPR * W;
    if ((threadIdx.x & 63) == 0) {
      lds[phase][0][w] = a;
      lds[phase][1][w] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += lds[phase][0][w0 + i];
      b += lds[phase][1][w0 + i];
    }
  }
}

// ---------------------------------------------------------------- forward
// The variance is summed from centred values (a second pass over the registers), so a mean
// far above the deviation cancels nothing.
template <typename T, int LPR, int NV>
__global__ void __launch_bounds__(kThreads<LPR>)
    k_norm_fwd(const T* __restrict__ X, const T* __restrict__ weight, const T* __restrict__ bias,
               int64_t rows, int n, int layer, float eps, T* __restrict__ Y,
               float* __restrict__ mean, float* __restrict__ rstd) {
  typedef typename Vec16<T>::type V;
  constexpr int VE = kVec<T>, RPB = kThreads<LPR> / LPR;
  __shared__ float lds[2][2][16];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  V w[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * LPR) * VE;
    w[i] = load_vec(weight, c, n);
    b[i] = V{};
    if (bias != nullptr) b[i] = load_vec(bias, c, n);
  }
  const float inv_n = 1.f / (float)n;
  int phase = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + sub;
    const bool on = row < rows;
    const T* x = X + (on ? row : 0) * n;
    float v[NV][VE];
    float s = 0.f, dummy = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const V t = load_vec(x, (lane + i * LPR) * VE, n);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        v[i][j] = (float)t[j];
        s += v[i][j];
      }
    }
    float mu = 0.f;
    if (layer) {
      row_sums<LPR>(s, dummy, lds, phase);
      phase ^= 1;
      mu = s * inv_n;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * LPR) * VE;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        v[i][j] = c + j < n ? v[i][j] - mu : 0.f;
        q += v[i][j] * v[i][j];
      }
    }
    row_sums<LPR>(q, dummy, lds, phase);
    phase ^= 1;
    const float r = 1.f / sqrtf(q * inv_n + eps);
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      V o;
#pragma unroll
      for (int j = 0; j < VE; ++j) o[j] = (T)(v[i][j] * r * (float)w[i][j] + (float)b[i][j]);
      store_vec(Y + row * n, (lane + i * LPR) * VE, n, o);
    }
    if (lane == 0) {
      if (layer) mean[row] = mu;
      rstd[row] = r;
    }
  }
}

// Rows too long for the registers of one block: the same sums in three passes over the row,
// the second and third of which come from L2.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_norm_fwd_long(const T* __restrict__ X, const T* __restrict__ weight,
                    const T* __restrict__ bias, int64_t rows, int n, int layer, float eps,
                    T* __restrict__ Y, float* __restrict__ mean, float* __restrict__ rstd) {
  typedef typename Vec16<T>::type V;
  constexpr int VE = kVec<T>;
  __shared__ float lds[2][2][16];
  const float inv_n = 1.f / (float)n;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = X + row * n;
    float s = 0.f, q = 0.f, dummy = 0.f;
    for (int c = threadIdx.x * VE; c < n; c += 1024 * VE) {
      const V t = load_vec(x, c, n);
#pragma unroll
      for (int j = 0; j < VE; ++j) s += (float)t[j];
    }
    row_sums<1024>(s, dummy, lds, 0);
    const float mu = layer ? s * inv_n : 0.f;
    for (int c = threadIdx.x * VE; c < n; c += 1024 * VE) {
      const V t = load_vec(x, c, n);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float d = c + j < n ? (float)t[j] - mu : 0.f;
        q += d * d;
      }
    }
    row_sums<1024>(q, dummy, lds, 1);
    const float r = 1.f / sqrtf(q * inv_n + eps);
    for (int c = threadIdx.x * VE; c < n; c += 1024 * VE) {
      const V t = load_vec(x, c, n), w = load_vec(weight, c, n);
      V b = {}, o;
      if (bias != nullptr) b = load_vec(bias, c, n);
#pragma unroll
      for (int j = 0; j < VE; ++j) o[j] = (T)(((float)t[j] - mu) * r * (float)w[j] + (float)b[j]);
      store_vec(Y + row * n, c, n, o);
    }
    if (threadIdx.x == 0) {
      if (layer) mean[row] = mu;
      rstd[row] = r;
    }
  }
}

// ---------------------------------------------------------------- backward
// Each block walks rows blockIdx, blockIdx + grid, ... (neighbouring blocks on neighbouring rows:
// with a run of rows for each block 32768 x 1536 took 7 % longer).  A lane holds the same columns of
// every row, so the weight's and bias's gradients add up in its registers; at the end the
// block's row groups are joined (lanes, then waves) into one partial row of dw and of db,
// which k_norm_reduce sums in block order.
template <typename T, int LPR, int NV, bool DB>
__global__ void __launch_bounds__(kThreadsBwd<LPR>, LPR == 256 ? 4 : 1)
    k_norm_bwd(const T* __restrict__ dY, const T* __restrict__ X, const T* __restrict__ weight,
               const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows, int n,
               T* __restrict__ dX, float* __restrict__ part_w, float* __restrict__ part_b) {
  typedef typename Vec16<T>::type V;
  constexpr int VE = kVec<T>, RPB = kThreadsBwd<LPR> / LPR;
  __shared__ float lds[2][2][16];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  V w[NV];
  float aw[NV][VE], ab[NV][VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = load_vec(weight, (lane + i * LPR) * VE, n);
#pragma unroll
    for (int j = 0; j < VE; ++j) aw[i][j] = ab[i][j] = 0.f;
  }
  const float inv_n = 1.f / (float)n;
  int phase = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < rows; row0 += (int64_t)gridDim.x * RPB) {
    const bool on = row0 + sub < rows;
    const int64_t row = on ? row0 + sub : rows - 1;
    // a row group past the end reads the last row and adds nothing
    const float r = rstd[row];
    const float mu = mean != nullptr ? mean[row] : 0.f;
    V x[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = fetch_vec(X + row * n, (lane + i * LPR) * VE, n);
      d[i] = fetch_vec(dY + row * n, (lane + i * LPR) * VE, n);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = place_vec<T>(x[i], (lane + i * LPR) * VE, n);
      d[i] = place_vec<T>(d[i], (lane + i * LPR) * VE, n);
    }
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float xh = ((float)x[i][j] - mu) * r, dy = (float)d[i][j], g = dy * (float)w[i][j];
        // columns at n and behind it have dy = 0 and w = 0, but (0 - mu) r may leave float32's range
        // (a test of xh itself would keep two of them: 40 % slower at 1536 columns)
        const float with = c1 + g * xh;
        c1 = (lane + i * LPR) * VE + j < n ? with : c1;
        c2 += g;
        if (on) {
          aw[i][j] += dy * xh;
          if (DB) ab[i][j] += dy;
        }
      }
    row_sums<LPR>(c1, c2, lds, phase);
    phase ^= 1;
    c1 *= inv_n;
    c2 = mean != nullptr ? c2 * inv_n : 0.f;
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      V o;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float xh = ((float)x[i][j] - mu) * r;
        o[j] = (T)(r * ((float)d[i][j] * (float)w[i][j] - c2 - xh * c1));
      }
      store_vec(dX + row * n, (lane + i * LPR) * VE, n, o);
    }
  }

  // the block's partial: lanes that hold the same columns are LPR apart
  if constexpr (LPR < 64) {
#pragma unroll
    for (int o = 32; o >= LPR; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          aw[i][j] += __shfl_xor(aw[i][j], o, 64);
          if (DB) ab[i][j] += __shfl_xor(ab[i][j], o, 64);
        }
  }
  constexpr int HOLD = LPR < 64 ? 64 : LPR, GROUPS = kThreadsBwd<LPR> / HOLD;
  if constexpr (GROUPS > 1) {
    __shared__ float joined[GROUPS - 1][NV * VE * LPR];
    const int group = threadIdx.x / HOLD;
    const bool mine = (int)threadIdx.x % HOLD < LPR;
    for (int pass = 0; pass < (DB ? 2 : 1); ++pass) {
      if (pass) __syncthreads();
      if (mine && group > 0)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VE; ++j)
            joined[group - 1][(i * VE + j) * LPR + lane] = pass ? ab[i][j] : aw[i][j];
      __syncthreads();
      if (mine && group == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            float t = pass ? ab[i][j] : aw[i][j];
#pragma unroll
            for (int k = 0; k < GROUPS - 1; ++k) t += joined[k][(i * VE + j) * LPR + lane];
            if (pass) ab[i][j] = t;
            else aw[i][j] = t;
          }
    }
    if (group != 0 || !mine) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    typedef __attribute__((ext_vector_type(4), aligned(4))) float F4;
    const int c = (lane + i * LPR) * VE;
#pragma unroll
    for (int j = 0; j < VE; j += 4) {
      store_vec(part_w + (int64_t)blockIdx.x * n, c + j, n,
                F4{aw[i][j], aw[i][j + 1], aw[i][j + 2], aw[i][j + 3]});
      if (DB)
        store_vec(part_b + (int64_t)blockIdx.x * n, c + j, n,
                  F4{ab[i][j], ab[i][j + 1], ab[i][j + 2], ab[i][j + 3]});
    }
  }
}

// Long rows: dx with two passes over the row; the columns' sums in a kernel of their own.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_norm_bwd_long(const T* __restrict__ dY, const T* __restrict__ X,
                    const T* __restrict__ weight, const float* __restrict__ mean,
                    const float* __restrict__ rstd, int64_t rows, int n, T* __restrict__ dX) {
  typedef typename Vec16<T>::type V;
  constexpr int VE = kVec<T>;
  __shared__ float lds[2][2][16];
  const float inv_n = 1.f / (float)n;
  int phase = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float r = rstd[row], mu = mean != nullptr ? mean[row] : 0.f;
    float c1 = 0.f, c2 = 0.f;
    for (int c = threadIdx.x * VE; c < n; c += 1024 * VE) {
      const V x = load_vec(X + row * n, c, n), d = load_vec(dY + row * n, c, n),
              w = load_vec(weight, c, n);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float g = (float)d[j] * (float)w[j];
        c1 += g * ((float)x[j] - mu) * r;
        c2 += g;
      }
    }
    row_sums<1024>(c1, c2, lds, phase);
    phase ^= 1;
    c1 *= inv_n;
    c2 = mean != nullptr ? c2 * inv_n : 0.f;
    for (int c = threadIdx.x * VE; c < n; c += 1024 * VE) {
      const V x = load_vec(X + row * n, c, n), d = load_vec(dY + row * n, c, n),
              w = load_vec(weight, c, n);
      V o;
#pragma unroll
      for (int j = 0; j < VE; ++j)
        o[j] = (T)(r * ((float)d[j] * (float)w[j] - c2 - ((float)x[j] - mu) * r * c1));
      store_vec(dX + row * n, c, n, o);
    }
  }
}

// One thread per column; block (x, y) sums rows y, y + gridDim.y, ... into partial row y.
template <typename T>
__global__ void __launch_bounds__(256)
    k_norm_cols_long(const T* __restrict__ dY, const T* __restrict__ X,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows,
                     int n, float* __restrict__ part_w, float* __restrict__ part_b) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float mu = mean != nullptr ? mean[row] : 0.f;
    const float dy = (float)dY[row * n + c];
    aw += dy * (((float)X[row * n + c] - mu) * rstd[row]);
    ab += dy;
  }
  part_w[(int64_t)blockIdx.y * n + c] = aw;
  if (part_b != nullptr) part_b[(int64_t)blockIdx.y * n + c] = ab;
}

// out[c] = (or +=) the sum over the np partial rows, in a fixed order: 16 row lanes of 64 columns
// each.  blockIdx.y picks dw or db.
__global__ void __launch_bounds__(1024)
    k_norm_reduce(const float* __restrict__ part_w, const float* __restrict__ part_b, int np, int n,
                  int accumulate, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float lds[16][64];
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? db : dw;
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int rl = threadIdx.x >> 6;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int p = rl; p < np; p += 16) s += part[(int64_t)p * n + c];
  }
  lds[rl][threadIdx.x & 63] = s;
  __syncthreads();
  if (rl == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += lds[i][threadIdx.x];
    out[c] = accumulate ? out[c] + s : s;
  }
}

// ---------------------------------------------------------------- launches
// How a row of n elements is held: lanes per row, vectors per lane; {0, 0}: long rows.  The
// fewest lanes that hold it in at most two vectors each (four for the longest rows).
struct RowShape {
  int lpr, nv;
};
template <typename T> RowShape row_shape(int64_t n, bool backward, bool bias) {
  static const RowShape shapes[] = {{4, 1},   {16, 1},  {64, 1},  {64, 2},  {256, 1},
                                    {256, 2}, {512, 2}, {512, 4}, {1024, 4}};
  for (const RowShape& s : shapes) {
    if (n > (int64_t)s.lpr * s.nv * kVec<T> || (s.lpr == 1024 && sizeof(T) != 4)) continue;
    // The backward of 16-bit rows that nearly fill 512 lanes of one vector is faster in those, with
    // fewer registers (32768 x 4096 with bias 147 us against 180), that of shorter rows in 256 lanes
    // of two, which keep more rows in flight (32768 x 2064, 2880 and 3328 without bias: 92, 110 and
    // 128 us against 119, 124 and 128).  The sums of a bias would not fit the registers of these: with
    // bias, 512 lanes at any length (151, 159 and 166 us against 123, 129 and 135).
    if (backward && sizeof(T) == 2 && s.lpr == 256 && s.nv == 2 && (bias || n > 416 * kVec<T>)) return {512, 1};
    return s;
  }
  return {0, 0};
}

#define GRPO_ROW_SHAPES(CASE) \
  CASE(4, 1) CASE(16, 1) CASE(64, 1) CASE(64, 2) CASE(256, 1) CASE(256, 2) CASE(512, 2) CASE(512, 4)

// Blocks of the backward, each of which leaves one partial row: as many as keep the loads
// going, but no more, since partial rows are written and read again (and the sums of a bias
// take registers: with three blocks a CU, 32768 x 2048 took 89 us, with two 77).  Long rows: as
// many as make 64 MB at most.
int64_t bwd_blocks(int64_t rows, int64_t n, RowShape sh, bool bias) {
  if (sh.lpr == 0) return std::min<int64_t>(rows, std::max<int64_t>(1, std::min<int64_t>(64, (1 << 24) / n)));
  const int64_t rpb = sh.lpr >= 256 ? std::max(1, 512 / sh.lpr) : 256 / sh.lpr;
  const int64_t most = sh.nv == 4 ? 1 : sh.lpr == 256 && sh.nv == 1 ? (bias ? 2 : 3) : sh.lpr >= 256 ? 2 : 4;
  return std::min<int64_t>((rows + rpb - 1) / rpb, most * kCUs);
}

template <typename T>
hipError_t launch_norm_fwd(const T* X, const T* w, const T* b, int64_t rows, int n, int layer,
                           float eps, T* Y, float* mean, float* rstd, hipStream_t s) {
  ScopedKernelTimer t(KK_NORM_FWD, s);
  const RowShape sh = row_shape<T>(n, false, b != nullptr);
  const int64_t rpb = sh.lpr == 0 ? 1 : std::max(1, 256 / sh.lpr);
  const unsigned grid = (unsigned)std::min<int64_t>((rows + rpb - 1) / rpb, 8 * kCUs);
#define GRPO_CASE(L, N)                                                                      \
  if (sh.lpr == L && sh.nv == N) {                                                           \
    k_norm_fwd<T, L, N><<<grid, kThreads<L>, 0, s>>>(X, w, b, rows, n, layer, eps, Y, mean, rstd); \
    return hipGetLastError();                                                                \
  }
  GRPO_ROW_SHAPES(GRPO_CASE)
  if constexpr (sizeof(T) == 4) {  // 16-bit rows that long would need twice the registers a lane
    GRPO_CASE(1024, 4)
  }
#undef GRPO_CASE
  k_norm_fwd_long<T><<<grid, 1024, 0, s>>>(X, w, b, rows, n, layer, eps, Y, mean, rstd);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_bwd(const T* dY, const T* X, const T* w, const float* mean,
                           const float* rstd, int64_t rows, int n, T* dX, float* part_w,
                           float* part_b, hipStream_t s) {
  ScopedKernelTimer t(KK_NORM_BWD, s);
  const RowShape sh = row_shape<T>(n, true, part_b != nullptr);
  const unsigned grid = (unsigned)bwd_blocks(rows, n, sh, part_b != nullptr);
#define GRPO_CASE(L, N)                                                                         \
  if (sh.lpr == L && sh.nv == N) {                                                              \
    if (part_b == nullptr)                                                                      \
      k_norm_bwd<T, L, N, false><<<grid, kThreadsBwd<L>, 0, s>>>(dY, X, w, mean, rstd, rows, n, dX, \
                                                              part_w, part_b);                  \
    else if constexpr (sizeof(T) == 4 || L != 256 || N != 2)                                    \
      k_norm_bwd<T, L, N, true><<<grid, kThreadsBwd<L>, 0, s>>>(dY, X, w, mean, rstd, rows, n, dX, \
                                                             part_w, part_b);                   \
    return hipGetLastError();                                                                   \
  }
  GRPO_ROW_SHAPES(GRPO_CASE)
  if constexpr (sizeof(T) == 4) {
    // 128 registers do not hold these rows (100 spill, with bias 116), but the long rows' passes take
    // longer: 4096 x 16384 176 us, 210 with bias, against 295 and 298 (512 rows: 42 and 52 against 39
    // and 40).  The 16-bit form of 512 lanes with four vectors and bias spills 16 (8192 x 12288: 136 us,
    // 4.4 TB/s).
    GRPO_CASE(1024, 4)
  } else {
    GRPO_CASE(512, 1)
  }
#undef GRPO_CASE
  k_norm_bwd_long<T><<<(unsigned)std::min<int64_t>(rows, 4 * kCUs), 1024, 0, s>>>(
      dY, X, w, mean, rstd, rows, n, dX);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_norm_cols_long<T><<<dim3((unsigned)((n + 255) / 256), grid), 256, 0, s>>>(
      dY, X, mean, rstd, rows, n, part_w, part_b);
  return hipGetLastError();
}

hipError_t launch_norm_reduce(const float* part_w, const float* part_b, int np, int n,
                              int accumulate, float* dw, float* db, hipStream_t s) {
  ScopedKernelTimer t(KK_NORM_REDUCE, s);
  k_norm_reduce<<<dim3((unsigned)((n + 63) / 64), db != nullptr ? 2 : 1), 1024, 0, s>>>(
      part_w, part_b, np, n, accumulate, dw, db);
  return hipGetLastError();
}

constexpr int64_t kMaxCols = 1 << 24;

int check_norm(int64_t rows, int64_t cols, int dtype, int kind) {
  if (rows <= 0 || cols <= 0)
    return fail(GRPO_ERR_INVALID_ARG, "rows and cols must be positive (rows=%lld cols=%lld)",
                (long long)rows, (long long)cols);
  if (dtype != GRPO_F32 && dtype != GRPO_BF16)
    return fail(GRPO_ERR_INVALID_ARG, "dtype %d is neither GRPO_F32 nor GRPO_BF16", dtype);
  if (kind != GRPO_NORM_LAYER && kind != GRPO_NORM_RMS)
    return fail(GRPO_ERR_INVALID_ARG, "norm kind %d is not 0 or 1", kind);
  if (rows > INT32_MAX || cols > kMaxCols)
    return fail(GRPO_ERR_UNSUPPORTED, "rows must fit int32 and cols be at most 2^24");
  return GRPO_OK;
}

// The number of partial rows for either type (their vectors differ, so their lanes do).
int64_t partial_rows(int64_t rows, int64_t cols, int dtype, bool bias) {
  return bwd_blocks(rows, cols, dtype == GRPO_F32 ? row_shape<float>(cols, true, bias) : row_shape<__bf16>(cols, true, bias),
                    bias);
}

}  // namespace
}  // namespace grpo

using grpo::fail;

extern "C" {

size_t grpo_norm_workspace_bytes(int64_t rows, int64_t cols, int dtype) {
  if (grpo::check_norm(rows, cols, dtype, GRPO_NORM_LAYER) != GRPO_OK) return 0;
  // either form may have more
  const int64_t most = std::max(grpo::partial_rows(rows, cols, dtype, false),
                                grpo::partial_rows(rows, cols, dtype, true));
  return 2 * grpo::align_up((size_t)(most * cols) * 4);
}

int grpo_norm_fwd(const void* X, const void* weight, const void* bias, int64_t rows, int64_t cols,
                  int dtype, int kind, float eps, void* Y, float* mean, float* rstd, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(X);
  GRPO_CHECK_PTR(weight);
  GRPO_CHECK_PTR(Y);
  GRPO_CHECK_PTR(rstd);
  const int st = grpo::check_norm(rows, cols, dtype, kind);
  if (st != GRPO_OK) return st;
  const int layer = kind == GRPO_NORM_LAYER;
  if (layer) GRPO_CHECK_PTR(mean);
  if (!isfinite(eps) || eps < 0.f)
    return fail(GRPO_ERR_INVALID_ARG, "eps must be finite and >= 0, not %g", (double)eps);
  if (Y == X) return fail(GRPO_ERR_INVALID_ARG, "Y may not be X");
  hipStream_t s = (hipStream_t)stream;
  if (dtype == GRPO_BF16)
    GRPO_HIP(grpo::launch_norm_fwd<__bf16>((const __bf16*)X, (const __bf16*)weight,
                                           (const __bf16*)bias, rows, (int)cols, layer, eps,
                                           (__bf16*)Y, mean, rstd, s));
  else
    GRPO_HIP(grpo::launch_norm_fwd<float>((const float*)X, (const float*)weight,
                                          (const float*)bias, rows, (int)cols, layer, eps,
                                          (float*)Y, mean, rstd, s));
  return GRPO_OK;
}

int grpo_norm_bwd(const void* dY, const void* X, const void* weight, const float* mean,
                  const float* rstd, int64_t rows, int64_t cols, int dtype, int kind,
                  int accumulate, void* dX, float* dweight, float* dbias, void* workspace,
                  size_t workspace_bytes, void* stream) {
  grpo::clear_error();
  GRPO_CHECK_PTR(dY);
  GRPO_CHECK_PTR(X);
  GRPO_CHECK_PTR(weight);
  GRPO_CHECK_PTR(rstd);
  GRPO_CHECK_PTR(dX);
  GRPO_CHECK_PTR(dweight);
  const int st = grpo::check_norm(rows, cols, dtype, kind);
  if (st != GRPO_OK) return st;
  const float* mu = kind == GRPO_NORM_LAYER ? mean : nullptr;
  if (kind == GRPO_NORM_LAYER) GRPO_CHECK_PTR(mean);
  if (accumulate != 0 && accumulate != 1)
    return fail(GRPO_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  const size_t need = grpo_norm_workspace_bytes(rows, cols, dtype);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(GRPO_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need,
                workspace == nullptr ? (size_t)0 : workspace_bytes);
  if ((uintptr_t)workspace % grpo::kAlign != 0)
    return fail(GRPO_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  // long rows are read again, for dweight, after dX is written
  if (dX == dY || dX == X) return fail(GRPO_ERR_INVALID_ARG, "dX may not be dY or X");
  hipStream_t s = (hipStream_t)stream;
  float* part_w = (float*)workspace;
  float* part_b = dbias == nullptr ? nullptr : (float*)((char*)workspace + need / 2);
  const int np = (int)grpo::partial_rows(rows, cols, dtype, dbias != nullptr);
  if (dtype == GRPO_BF16)
    GRPO_HIP(grpo::launch_norm_bwd<__bf16>((const __bf16*)dY, (const __bf16*)X,
                                           (const __bf16*)weight, mu, rstd, rows, (int)cols,
                                           (__bf16*)dX, part_w, part_b, s));
  else
    GRPO_HIP(grpo::launch_norm_bwd<float>((const float*)dY, (const float*)X, (const float*)weight,
                                          mu, rstd, rows, (int)cols, (float*)dX, part_w, part_b,
                                          s));
  GRPO_HIP(grpo::launch_norm_reduce(part_w, part_b, np, (int)cols, accumulate, dweight, dbias, s));
  return GRPO_OK;
}

}  // extern "C"
