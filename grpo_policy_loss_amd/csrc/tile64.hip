// tile64.hip -- the log-probabilities' products in 64 x 64 tiles: float32, and bfloat16
// gradients of few tokens or a small head, where 256 x 256 tiles leave most of the chip idle.
//
//   k64_lse     z = W_tile . H_tile^T folded into (max, sum exp) per token and 64 vocabulary rows
//   k64_merge   those of a token joined: lp and lse
//   k64_dz      the same tile recomputed: dZ[t][v] = g_t (onehot - softmax) dz/d(w h), stored
//               [tokens][vocabulary] in H's type
//   k64_grads   one launch for both gradients: dH[t][:] = sum_v dZ[t][v] W[v][:] (in shares of
//               the vocabulary where that alone has few tiles) and dW[v][:] = sum_t dZ[t][v] h_t
//   k64_join    the sum of the shares
// Two and two or three launches in place of two and nine: tokens without a gradient are not packed away, their rows of
// dZ are 0 (their hidden states, which may hold anything, are read as 0), and both gradients are
// written where they belong.
//
// A block is 4 waves, each 32 x 32 of the tile in 2 x 2 blocks of the 16 x 16 matrix
// instruction; or, of a 32 x 32 tile (M = 32), one such block each, where 64 x 64 tiles would not
// give every CU one or tokens fill no more than half of one.  K advances by 64; each step's tiles go through registers into one of two LDS
// slots, read two steps ahead of their use.  An operand may lie K-major (the elements of one k
// adjacent): its 4 x 4 blocks are transposed in registers on their way, so that fragments are 16
// adjacent bytes of a row in either case.
#include <math.h>

#include <algorithm>

#include "elem.hpp"
#include "kernels.hpp"
#include "raster.hpp"
#include "timing.hpp"

namespace grpo {
namespace {

typedef __attribute__((ext_vector_type(4))) float f4;
typedef __attribute__((ext_vector_type(8))) __bf16 b8;
typedef __attribute__((ext_vector_type(4))) __bf16 b4;

constexpr int kK = 64;         // k of a step
constexpr int kThreads64 = 256;

// LDS rows of 64 k, padded so that 16 rows at one k spread over the banks.
template <typename T> constexpr int kPitch = sizeof(T) == 4 ? 68 : 72;
template <typename T, int M> constexpr int kSlot = M * kPitch<T>;   // elements of one operand's slot

template <typename T> struct Four;
template <> struct Four<float> {
  typedef __attribute__((ext_vector_type(4), aligned(4))) float type;
};
template <> struct Four<__bf16> {
  typedef __attribute__((ext_vector_type(4), aligned(2))) __bf16 type;
};

// One operand: element (r, k) at p[r ld + k], or at p[k ld + r] if K-major, for r < rows and
// k < k_end; anything else reads as 0.  Rows and, unless K-major, k come in whole vectors.
// gate (K-major): k with gate[k] = 0 read as 0 too.
template <typename T>
struct Side {
  const T* p;
  int64_t ld;
  int rows, k_end;
  const float* gate;
};

// A thread's share of an operand's M x 64 tile at (r0, k0): a 4 x 4 block if K-major (the first
// 4 M threads have one), else M / 4 elements.
template <typename T, bool KM, int M>
struct Share {
  static constexpr int kWide = KM ? 4 : 16 / (int)sizeof(T);     // elements of a load
  static constexpr int kLoads = KM ? 4 : M / 4 / kWide;
  typedef typename std::conditional<kWide == 8, typename Vec16<__bf16>::type, typename Four<T>::type>::type V;
  V v[kLoads];
  float g[4];
  unsigned ok;

  __device__ __forceinline__ void load(const Side<T>& s, int r0, int k0) {
    ok = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int r, k;
      place(i, r, k);
      const bool in = r0 + r < s.rows && k0 + k < s.k_end && k < kK;
      const int64_t at = KM ? (int64_t)(k0 + k) * s.ld + r0 + r : (int64_t)(r0 + r) * s.ld + k0 + k;
      v[i] = *(const V*)(s.p + (in ? at : 0));
      ok |= (unsigned)in << i;
      if (KM && s.gate != nullptr) g[i] = s.gate[in ? k0 + k : 0];
      else g[i] = 1.f;
    }
  }
  // Row and k of load i within the tile.
  static __device__ __forceinline__ void place(int i, int& r, int& k) {
    const int t = threadIdx.x;
    if (KM) r = 4 * (t & (M / 4 - 1)), k = 4 * (t / (M / 4)) + i;
    else if (kWide == 4) r = (t >> 4) + 16 * i, k = 4 * (t & 15);
    else r = (t >> 3) + 32 * i, k = 8 * (t & 7);
  }
  __device__ __forceinline__ void store(T* lds) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (!(ok >> i & 1) || g[i] == 0.f) v[i] = V{};
    if constexpr (KM) {
      int r, k;
      place(0, r, k);
      if (k >= kK) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        typedef __attribute__((ext_vector_type(4))) T W;
        *(W*)(lds + (r + j) * kPitch<T> + k) = W{v[0][j], v[1][j], v[2][j], v[3][j]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        int r, k;
        place(i, r, k);
        typedef __attribute__((ext_vector_type(kWide))) T W;
        *(W*)(lds + r * kPitch<T> + k) = (W)v[i];
      }
    }
  }
};

// Blocks of a wave in each direction, and its accumulators.
template <int M> constexpr int kB = M / 32;
template <int M> using AccM = f4[kB<M>][kB<M>];

// One step's products from LDS.
template <typename T, int M>
__device__ __forceinline__ void step64(AccM<M>& acc, const T* a, const T* b) {
  constexpr int B = kB<M>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, g = lane >> 4;
  const T* ar = a + ((wave >> 1) * (M / 2) + row) * kPitch<T>;
  const T* br = b + ((wave & 1) * (M / 2) + row) * kPitch<T>;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f4 x[B], y[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        x[i] = *(const f4*)(ar + 16 * i * kPitch<T> + 16 * s + 4 * g);
        y[i] = *(const f4*)(br + 16 * i * kPitch<T> + 16 * s + 4 * g);
      }
      // instruction e takes element e of every lane: 4 of the 16 k, the same for both sides
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
          for (int j = 0; j < B; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i][e], y[j][e], acc[i][j], 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      b8 x[B], y[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        x[i] = *(const b8*)(ar + 16 * i * kPitch<T> + 32 * s + 8 * g);
        y[i] = *(const b8*)(br + 16 * i * kPitch<T> + 32 * s + 8 * g);
      }
#pragma unroll
      for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
    }
  }
}

// acc = sum over k in [k0, k1) of A[ra + m][k] B[rb + n][k].  lds: 4 slots.
template <typename T, bool AKM, bool BKM, int M>
__device__ __forceinline__ void tile64(AccM<M>& acc, const Side<T>& A, int ra, const Side<T>& B, int rb,
                                       int k0, int k1, T* lds) {
#pragma unroll
  for (int i = 0; i < kB<M>; ++i)
#pragma unroll
    for (int j = 0; j < kB<M>; ++j) acc[i][j] = f4{};
  const int steps = (k1 - k0 + kK - 1) / kK;
  if (steps <= 0) return;
  Share<T, AKM, M> a0, a1;
  Share<T, BKM, M> b0, b1;
  a0.load(A, ra, k0);
  b0.load(B, rb, k0);
  if (steps > 1) {
    a1.load(A, ra, k0 + kK);
    b1.load(B, rb, k0 + kK);
  }
  a0.store(lds);
  b0.store(lds + kSlot<T, M>);
  // no load here is under a condition, so that a wait for the older ones does not wait for the newer
  int s = 0;
  for (; s + 3 < steps; s += 2) {
    a0.load(A, ra, k0 + (s + 2) * kK);
    b0.load(B, rb, k0 + (s + 2) * kK);
    __syncthreads();                       // slot 0 is written, slot 1 has been read
    step64<T, M>(acc, lds, lds + kSlot<T, M>);
    a1.store(lds + 2 * kSlot<T, M>);
    b1.store(lds + 3 * kSlot<T, M>);
    a1.load(A, ra, k0 + (s + 3) * kK);
    b1.load(B, rb, k0 + (s + 3) * kK);
    __syncthreads();
    step64<T, M>(acc, lds + 2 * kSlot<T, M>, lds + 3 * kSlot<T, M>);
    a0.store(lds);
    b0.store(lds + kSlot<T, M>);
  }
  // one to three steps are left: s in slot 0, s + 1 on its way
  if (s + 2 < steps) {
    a0.load(A, ra, k0 + (s + 2) * kK);
    b0.load(B, rb, k0 + (s + 2) * kK);
  }
  __syncthreads();
  step64<T, M>(acc, lds, lds + kSlot<T, M>);
  if (s + 1 >= steps) return;
  a1.store(lds + 2 * kSlot<T, M>);
  b1.store(lds + 3 * kSlot<T, M>);
  __syncthreads();
  step64<T, M>(acc, lds + 2 * kSlot<T, M>, lds + 3 * kSlot<T, M>);
  if (s + 2 >= steps) return;
  a0.store(lds);
  b0.store(lds + kSlot<T, M>);
  __syncthreads();
  step64<T, M>(acc, lds, lds + kSlot<T, M>);
}

// Row (of A) of element 0 of block i, and column (of B) of block j, of this lane in the tile; the
// elements of a block are 4 adjacent rows.
template <int M>
__device__ __forceinline__ int row_of(int i) {
  return (int)(threadIdx.x >> 7) * (M / 2) + 16 * i + 4 * ((int)(threadIdx.x & 63) >> 4);
}
template <int M>
__device__ __forceinline__ int col_of(int j) {
  return (int)(threadIdx.x >> 6 & 1) * (M / 2) + 16 * j + (int)(threadIdx.x & 15);
}

// Tile of workgroup bid: hardware deals workgroups to the 8 XCDs in turn; each gets a contiguous
// range of the raster, in groups of 8 row tiles, so that its L2 holds the panels they share.
__device__ __forceinline__ bool tile_of(int bid, int tm, int tn, int& mt, int& nt) {
  const int tiles = tm * tn, per = (tiles + 7) / 8;
  const int p = (bid & 7) * per + (bid >> 3);
  if ((bid >> 3) >= per || p >= tiles) return false;
  group_coords<8>(p, tm, tn, mt, nt);
  return true;
}
inline int64_t tile_grid(int64_t tiles) { return (tiles + 7) / 8 * 8; }

// The transformed logit and its slope.
__device__ __forceinline__ float transform(float z, const LogitXform& xf, float& slope) {
  if (!xf.softcap) {
    slope = xf.k;
    return xf.k * z;
  }
  const float t = tanhf(xf.a * z);
  slope = xf.a * xf.b * (1.f - t * t);
  return xf.b * t;
}

// A = W (rows: vocabulary), B = H (columns: tokens), K = d.
template <typename T, int M>
__global__ void __launch_bounds__(kThreads64)
    k64_lse(const T* __restrict__ W, const T* __restrict__ H, const int32_t* __restrict__ y, int V,
            int d, int C, int tm, int tn, LogitXform xf, float* __restrict__ part_m,
            float* __restrict__ part_s, float* __restrict__ zy) {
  __shared__ __attribute__((aligned(16))) T lds[4 * kSlot<T, M>];
  int mt, nt;
  if (!tile_of(blockIdx.x, tm, tn, mt, nt)) return;
  const int v0 = mt * M, t0 = nt * M;
  constexpr int B = kB<M>;
  int target[B];
#pragma unroll
  for (int j = 0; j < B; ++j) target[j] = t0 + col_of<M>(j) < C ? y[t0 + col_of<M>(j)] - v0 : -1;
  AccM<M> acc;
  tile64<T, false, false, M>(acc, Side<T>{W, d, V, d, nullptr}, v0, Side<T>{H, d, C, d, nullptr}, t0, 0, d, lds);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float mx[B], sum[B];
#pragma unroll
  for (int j = 0; j < B; ++j) {
    float z[4 * B], slope, m = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int v = row_of<M>(i) + e;
        const float x = transform(acc[i][j][e], xf, slope);
        z[4 * i + e] = v0 + v < V ? x : -__builtin_huge_valf();
        if (v == target[j] && v0 + v < V && t0 + col_of<M>(j) < C) zy[t0 + col_of<M>(j)] = x;
        m = __builtin_elementwise_maximum(m, z[4 * i + e]);     // NaN stays
      }
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16, 64));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 32, 64));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * B; ++i) s += z[i] == -__builtin_huge_valf() ? 0.f : expf(z[i] - m);
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    mx[j] = m;
    sum[j] = s;
  }
  // the other half of the rows is in the wave two further on
  __syncthreads();
  float* red = (float*)lds;
  if (wave >= 2 && lane < 16) {
#pragma unroll
    for (int j = 0; j < B; ++j) {
      red[2 * col_of<M>(j)] = mx[j];
      red[2 * col_of<M>(j) + 1] = sum[j];
    }
  }
  __syncthreads();
  if (wave >= 2 || lane >= 16) return;
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int t = t0 + col_of<M>(j);
    if (t >= C) continue;
    const float m2 = red[2 * col_of<M>(j)], s2 = red[2 * col_of<M>(j) + 1];
    const float m = __builtin_elementwise_maximum(mx[j], m2);
    float s = 0.f;
    if (m != -__builtin_huge_valf()) s = sum[j] * expf(mx[j] - m) + s2 * expf(m2 - m);
    part_m[(int64_t)mt * C + t] = m;
    part_s[(int64_t)mt * C + t] = s;
  }
}

// 16 tokens a block, 16 threads each.  lse is M + log sum; lp comes from its parts, so that it does not
// carry the rounding of an lse that is much larger, and rest is what that rounding left.
__global__ void __launch_bounds__(256)
    k64_merge(const float* __restrict__ part_m, const float* __restrict__ part_s,
              const float* __restrict__ zy, const int32_t* __restrict__ y, int V, int tiles,
              int64_t stride, int C, float* __restrict__ lp, float* __restrict__ lse, float* __restrict__ rest) {
  __shared__ float sm[16][17];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4, t = blockIdx.x * 16 + c;
  const int at = min(t, C - 1);
  float m = -__builtin_huge_valf();
  for (int i = q; i < tiles; i += 16) m = __builtin_elementwise_maximum(m, part_m[i * stride + at]);
  sm[q][c] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k) m = __builtin_elementwise_maximum(m, sm[k][c]);
  float s = 0.f;
  for (int i = q; i < tiles; i += 16) {
    const float p = part_s[i * stride + at];
    if (p != 0.f) s += p * expf(part_m[i * stride + at] - m);
  }
  __syncthreads();
  sm[q][c] = s;
  __syncthreads();
  if (q != 0 || t >= C) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += sm[k][c];
  const float ls = logf(s), sum = m + ls, b = sum - m;
  lp[t] = y[t] >= 0 && y[t] < V ? (zy[t] - m) - ls : __builtin_nanf("");
  lse[t] = sum;
  rest[t] = (m - (sum - b)) + (ls - b);
}

template <typename T, int M>
__global__ void __launch_bounds__(kThreads64)
    k64_dz(const T* __restrict__ W, const T* __restrict__ H, const int32_t* __restrict__ y,
           const float* __restrict__ lp, const float* __restrict__ lse, const float* __restrict__ rest,
           const float* __restrict__ grad_lp, int V, int d, int C, int vpad, int tm, int tn,
           LogitXform xf, T* __restrict__ dZ) {
  __shared__ __attribute__((aligned(16))) T lds[4 * kSlot<T, M>];
  int mt, nt;
  if (!tile_of(blockIdx.x, tm, tn, mt, nt)) return;
  const int v0 = mt * M, t0 = nt * M;
  constexpr int B = kB<M>;
  float c[B], hi[B], lo[B], of[B];
  int target[B];
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int t = min(t0 + col_of<M>(j), C - 1);
    c[j] = t0 + col_of<M>(j) < C ? grad_lp[t] : 0.f;
    hi[j] = lse[t];
    lo[j] = rest != nullptr ? rest[t] : 0.f;
    of[j] = lp[t];
    target[j] = y[t] - v0;
  }
  AccM<M> acc = {};
  // tokens without any gradient: their rows are 0
  if (__syncthreads_or(c[0] != 0.f || c[B - 1] != 0.f))
    tile64<T, false, false, M>(acc, Side<T>{W, d, V, d, nullptr}, v0, Side<T>{H, d, C, d, nullptr}, t0, 0, d, lds);
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int t = t0 + col_of<M>(j);
    if (t >= C) continue;
    const float at_target = c[j] * -expm1f(of[j]);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int v = row_of<M>(i);
      typename Four<T>::type q;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float slope, x;
        const float z = transform(acc[i][j][e], xf, slope);
        // z - lse nearly cancels where it counts: what is left of lse in float32 comes after
        x = -c[j] * expf((z - hi[j]) - lo[j]);
        if (v + e == target[j]) x = at_target;
        q[e] = (T)(c[j] == 0.f || v0 + v + e >= V ? 0.f : x * slope);
      }
      *(typename Four<T>::type*)(dZ + (int64_t)t * vpad + v0 + v) = q;
    }
  }
}

// Workgroups [0, tm_h tn_h shares): dH; those behind: dW.
template <typename T, int M>
__global__ void __launch_bounds__(kThreads64)
    k64_grads(const T* __restrict__ W, const T* __restrict__ H, const T* __restrict__ dZ,
              const float* __restrict__ grad_lp, int V, int d, int C, int vpad, int h_grid, int shares,
              int share_v, T* __restrict__ dH, float* __restrict__ parts, int accumulate,
              int dw_bf16, void* __restrict__ dW) {
  __shared__ __attribute__((aligned(16))) T lds[4 * kSlot<T, M>];
  constexpr int B = kB<M>;
  const int tm = (d + M - 1) / M;
  int mt, nt;
  AccM<M> acc;
  if ((int)blockIdx.x < h_grid) {
    const int tn = (C + M - 1) / M;
    // the shares outermost: those of one are on one XCD and read the same rows of W
    if (!tile_of(blockIdx.x, tm, tn * shares, mt, nt)) return;
    const int share = nt / tn, n0 = mt * M, t0 = (nt - share * tn) * M;
    const int k0 = share * share_v, k1 = min(k0 + share_v, vpad);
    tile64<T, true, false, M>(acc, Side<T>{W, d, d, V, nullptr}, n0, Side<T>{dZ, vpad, C, vpad, nullptr}, t0, k0, k1, lds);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int t = t0 + col_of<M>(j);
      if (t >= C) continue;
      const bool none = grad_lp[t] == 0.f;      // 0 whatever W holds
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int n = n0 + row_of<M>(i);
        if (n >= d) continue;
        if (none) acc[i][j] = f4{};
        if (shares > 1) {
          *(f4*)(parts + ((int64_t)share * C + t) * d + n) = acc[i][j];
        } else {
          typename Four<T>::type q;
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = (T)acc[i][j][e];
          *(typename Four<T>::type*)(dH + (int64_t)t * d + n) = q;
        }
      }
    }
    return;
  }
  if (!tile_of(blockIdx.x - h_grid, tm, (V + M - 1) / M, mt, nt)) return;
  const int n0 = mt * M, v0 = nt * M;
  tile64<T, true, true, M>(acc, Side<T>{H, d, d, C, grad_lp}, n0, Side<T>{dZ, vpad, vpad, C, nullptr}, v0, 0, C, lds);
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int v = v0 + col_of<M>(j);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int n = n0 + row_of<M>(i);
      if (v >= V || n >= d) continue;
      if (dw_bf16) {
        typename Four<__bf16>::type q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = (__bf16)acc[i][j][e];
        *(typename Four<__bf16>::type*)((__bf16*)dW + (int64_t)v * d + n) = q;
      } else {
        typedef typename Four<float>::type V4;
        V4* to = (V4*)((float*)dW + (int64_t)v * d + n);
        *to = accumulate ? *to + (V4)acc[i][j] : (V4)acc[i][j];
      }
    }
  }
}

// dH = the sum of the shares, 4 elements a lane.
template <typename T>
__global__ void __launch_bounds__(256)
    k64_join(const float* __restrict__ parts, int shares, int64_t n, T* __restrict__ dH) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  f4 s = *(const f4*)(parts + at);
  for (int k = 1; k < shares; ++k) s += *(const f4*)(parts + k * n + at);
  typename Four<T>::type q;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = (T)s[e];
  *(typename Four<T>::type*)(dH + at) = q;
}

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

// 32 where 64 x 64 tiles would not give every CU one, or tokens (cols) would leave a quarter or more of
// theirs empty that 32 would not.  us of k64_dz, 64 against 32:
//   float32                   N = 3       64          300         3000
//   d 64,   V 1000             8   6       8   7       9   6       20  18
//   d 1024, V 64              30  13      30  14      30  14       32  14
//   d 1024, V 8000            30  14      32  20      74  66
//   d 4096, V 1000           100  38     102  38     103  57
//   d 1024, V 32000           48  30      51  54
//   bfloat16, d 4096, V 1000  29  20      30  20      30  23
int tile_rows(int64_t rows, int64_t cols) {
  const int64_t of64 = (cols + 63) / 64 * 64, of32 = (cols + 31) / 32 * 32;
  return (rows + 63) / 64 * (of64 / 64) < 256 || 4 * of32 <= 3 * of64 ? 32 : 64;
}

hipError_t launch64_lse(const float* W, const float* H, const int32_t* y, int64_t V, int64_t d, int C,
                        const LogitXform& xf, float* part_m, float* part_s, float* zy,
                        hipStream_t s) {
  ScopedKernelTimer timer(KK_LSE64, s);
  const int M = tile_rows(V, C), tm = cdiv(V, M), tn = cdiv(C, M);
  const auto k = M == 32 ? k64_lse<float, 32> : k64_lse<float, 64>;
  k<<<(unsigned)tile_grid((int64_t)tm * tn), kThreads64, 0, s>>>(W, H, y, (int)V, (int)d, C, tm, tn, xf, part_m, part_s,
                                                                zy);
  return hipGetLastError();
}

hipError_t launch64_merge(const float* part_m, const float* part_s, const float* zy,
                          const int32_t* y, int64_t V, int tiles, int64_t stride, int C, float* lp,
                          float* lse, float* rest, hipStream_t s) {
  ScopedKernelTimer timer(KK_MERGE64, s);
  k64_merge<<<cdiv(C, 16), 256, 0, s>>>(part_m, part_s, zy, y, (int)V, tiles, stride, C, lp, lse, rest);
  return hipGetLastError();
}

template <typename T>
hipError_t launch64_dz(const T* W, const T* H, const int32_t* y, const float* lp, const float* lse,
                       const float* rest, const float* grad_lp, int64_t V, int64_t d, int C,
                       int64_t vpad, const LogitXform& xf, T* dZ, hipStream_t s) {
  ScopedKernelTimer timer(KK_DZ64, s);
  // the tiles cover vpad: its columns from V on are read as 0
  const int M = tile_rows(V, C), tm = cdiv(vpad, M), tn = cdiv(C, M);
  const auto k = M == 32 ? k64_dz<T, 32> : k64_dz<T, 64>;
  k<<<(unsigned)tile_grid((int64_t)tm * tn), kThreads64, 0, s>>>(W, H, y, lp, lse, rest, grad_lp, (int)V, (int)d, C,
                                                                (int)vpad, tm, tn, xf, dZ);
  return hipGetLastError();
}

template <typename T>
hipError_t launch64_grads(const T* W, const T* H, const T* dZ, const float* grad_lp, int64_t V,
                          int64_t d, int C, int64_t vpad, int shares, T* dH, float* parts,
                          int accumulate, int dw_bf16, void* dW, hipStream_t s) {
  // 32 where dW has few tiles.  us, 64 against 32, float32: d 64, V 1000 (16 tiles) 14 and 9 of 300 tokens,
  // 89 and 68 of 3000; d 64, V 8000 (125) 15 and 18, 178 and 131; d 1024, V 1000 (256) 31 and 30,
  // 211 and 218; d 256, V 8000 (500) 39 and 52, 301 and 376
  const int M = (int64_t)cdiv(d, 64) * cdiv(V, 64) <= 128 ? 32 : 64, tm = cdiv(d, M);
  const int64_t h = dH != nullptr ? tile_grid((int64_t)tm * cdiv(C, M) * shares) : 0;
  const int64_t w = dW != nullptr ? tile_grid((int64_t)tm * cdiv(V, M)) : 0;
  {
    ScopedKernelTimer timer(KK_GRADS64, s);
    const int share_v = cdiv(vpad / kK, shares) * kK;
    const auto k = M == 32 ? k64_grads<T, 32> : k64_grads<T, 64>;
    k<<<(unsigned)(h + w), kThreads64, 0, s>>>(W, H, dZ, grad_lp, (int)V, (int)d, C, (int)vpad, (int)h, shares, share_v,
                                              dH, parts, accumulate, dw_bf16, dW);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dH == nullptr || shares == 1) return hipSuccess;
  ScopedKernelTimer timer(KK_JOIN64, s);
  const int64_t n = (int64_t)C * d;
  k64_join<T><<<cdiv(n, 1024), 256, 0, s>>>(parts, shares, n, dH);
  return hipGetLastError();
}

#define GRPO_INSTANTIATE64(T)                                                                     \
  template hipError_t launch64_dz<T>(const T*, const T*, const int32_t*, const float*,            \
                                     const float*, const float*, const float*, int64_t, int64_t,  \
                                     int, int64_t, const LogitXform&, T*, hipStream_t);           \
  template hipError_t launch64_grads<T>(const T*, const T*, const T*, const float*, int64_t,      \
                                        int64_t, int, int64_t, int, T*, float*, int, int, void*,  \
                                        hipStream_t);
GRPO_INSTANTIATE64(float)
GRPO_INSTANTIATE64(__bf16)

}  // namespace grpo
