// tile64.hip -- the log-probabilities' products in 64 x 64 tiles: float32, and bfloat16
// gradients of few tokens or a small head, where 256 x 256 tiles leave most of the chip idle.
//
//   k64_lse     z = W_tile . H_tile^T folded into (max, sum exp) per token and 64 vocabulary rows
//   k64_merge   those of a token joined: lp and lse
//   k64_dz      the same tile recomputed: dZ[t][v] = g_t (onehot - softmax) dz/d(w h), stored
//               [tokens][vocabulary] in H's type
//   k64_grads   one launch for both gradients: dH[t][:] = sum_v dZ[t][v] W[v][:] (in shares of
//               the vocabulary where that alone has few tiles) and dW[v][:] = sum_t dZ[t][v] h_t
//               (likewise in shares of the tokens)
//   k64_join    the sum of the shares
// Two and two or three launches in place of two and nine: tokens without a gradient are not packed
// away, their rows of dZ are 0 (their hidden states, which may hold anything, are read as 0), and both
// gradients are written where they belong.
//
// A block is 4 waves, each 32 x 32 of the tile in 2 x 2 blocks of the 16 x 16 matrix
// instruction; or, of a 32 x 32 tile (M = 32), one such block each, where 64 x 64 tiles would not
// give every CU one or tokens fill no more than half of one.  K advances by 64; each step's tiles go
// through registers into LDS, from loads that are one or two steps ahead of their use.  An operand may
// lie K-major (the elements of one k adjacent): its 4 x 4 blocks are transposed in registers on their
// way, so that fragments are 16 adjacent bytes of a row in either case.
//
// What bounds them: few tokens of a small head the latency of a step (1 us and less) times the steps;
// few tokens of a large head W's bytes; float32 else the matrix instructions, which at 157 TFLOP/s take 32
// cycles for 2048 operations and share their units with other vector arithmetic: there must be little
// of it, and four blocks a CU to take turns.  2048 tokens, d 1024, V 8000, float32: forward 287 us,
// 117 TFLOP/s (81 % of the matrix units' cycles), backward 870 us, 116.
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
// Slots of each operand.  float32 tiles of 64 take one, and a barrier more a step, so that 4 blocks fit a
// CU (34 KB; with two, 69 KB, 2 blocks): backward of 2048 tokens, d 1024, V 8000 945 against 1060 us.
template <typename T, int M> constexpr int kSlots = sizeof(T) == 4 && M == 64 ? 1 : 2;

template <typename T> struct Four;
template <> struct Four<float> {
  typedef __attribute__((ext_vector_type(4), aligned(4))) float type;
};
template <> struct Four<__bf16> {
  typedef __attribute__((ext_vector_type(4), aligned(2))) __bf16 type;
};

// One operand: element (r, k) at p[r ld + k], or at p[k ld + r] if K-major, for r < rows and
// k < k_end.  From k_end on it reads as 0; from rows on as some row (whose results are not kept).
// Rows and, unless K-major, k come in whole vectors.  gate: k with gate[k] = 0 read as 0 too.
template <typename T>
struct Side {
  const T* p;
  int64_t ld;
  int rows, k_end;
  const float* gate;
};

// A thread's share of an operand's M x 64 tile at row r0: a 4 x 4 block if K-major (the first 4 M
// threads have one), else M / 4 elements.  Its place in a step's tile stays, so that a step's loads
// take no arithmetic but a step of their scalar base: float32 products share their units with it.
template <typename T, bool KM, bool GATE, int M>
struct Share {
  static constexpr int kWide = KM ? 4 : 16 / (int)sizeof(T);     // elements of a load
  static constexpr int kLoads = KM ? 4 : M / 4 / kWide;
  typedef typename std::conditional<kWide == 8, typename Vec16<__bf16>::type, typename Four<T>::type>::type V;
  struct Step {
    V v[kLoads];
    typename Four<float>::type g;      // GATE: of the 4 k
  };
  const char* base;
  const float* gate;
  int64_t ld;
  int k_end, r, k;
  uint32_t off[kLoads];

  __device__ __forceinline__ Share(const Side<T>& s, int r0) : gate(s.gate), ld(s.ld), k_end(s.k_end) {
    // rows that lie behind the last read that one
    const int last = s.rows - (KM ? 4 : 1), first = min(r0, last);
    base = (const char*)(s.p + (KM ? (int64_t)first : first * s.ld));
    const int t = threadIdx.x;
    // float32: neighbours at 4 k and 4 r, whose writes so share no bank (4 rows of LDS are 16 banks apart)
    if (KM && sizeof(T) == 4) r = 4 * (t >> 2 & (M / 4 - 1)), k = 4 * (t & 3) + 16 * (t / M);
    else if (KM) r = 4 * (t & (M / 4 - 1)), k = 4 * (t / (M / 4));
    else if (kWide == 4) r = t >> 4, k = 4 * (t & 15);
    else r = t >> 3, k = 8 * (t & 7);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int ri = min(r + row_step() * i, last - first);
      off[i] = (uint32_t)(KM ? (int64_t)((k & (kK - 1)) + i) * ld + ri : ri * ld + k) * (uint32_t)sizeof(T);
    }
  }
  static constexpr int row_step() { return KM ? 0 : kWide == 4 ? 16 : 32; }
  __device__ __forceinline__ const char* at(int k0) const {
    return base + (KM ? k0 * ld : (int64_t)k0) * (int64_t)sizeof(T);
  }
  // The 64 k from k0 on, all below k_end.
  __device__ __forceinline__ void load(Step& x, int k0) const {
    const char* p = at(k0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x.v[i] = *(const V*)(p + off[i]);
    if (GATE) x.g = *(const typename Four<float>::type*)((const char*)(gate + k0) + 4u * (uint32_t)(k & (kK - 1)));
  }
  // Those there are.
  __device__ __forceinline__ void load_tail(Step& x, int k0) const {
    const char* p = at(k0);
    static_assert(!GATE || kLoads == 4, "a gate for each load");
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int ki = (k & (kK - 1)) + (KM ? i : 0);
      x.v[i] = V{};
      if (GATE) x.g[i] = 0.f;
      if (k0 + ki >= k_end) continue;
      x.v[i] = *(const V*)(p + off[i]);
      if (GATE) x.g[i] = gate[k0 + ki];
    }
  }
  __device__ __forceinline__ void store(Step& x, T* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (GATE && x.g[i] == 0.f) x.v[i] = V{};
    if constexpr (KM) {
      if (k >= kK) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        typedef __attribute__((ext_vector_type(4))) T W;
        *(W*)(lds + (r + j) * kPitch<T> + k) = W{x.v[0][j], x.v[1][j], x.v[2][j], x.v[3][j]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        typedef __attribute__((ext_vector_type(kWide))) T W;
        *(W*)(lds + (r + row_step() * i) * kPitch<T> + k) = (W)x.v[i];
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

// acc = sum over k in [k0, k1) of A[ra + m][k] B[rb + n][k].  lds: kSlots slots of each.
template <typename T, bool AKM, bool BKM, bool GATE, int M>
__device__ __forceinline__ void tile64(AccM<M>& acc, const Side<T>& A, int ra, const Side<T>& B, int rb,
                                       int k0, int k1, T* lds) {
  constexpr int kTwo = kSlot<T, M>;
#pragma unroll
  for (int i = 0; i < kB<M>; ++i)
#pragma unroll
    for (int j = 0; j < kB<M>; ++j) acc[i][j] = f4{};
  const int end = min(k1, min(A.k_end, B.k_end)), full = max(end - k0, 0) / kK;
  const Share<T, AKM, GATE, M> a(A, ra);
  const Share<T, BKM, false, M> b(B, rb);
  typename Share<T, AKM, GATE, M>::Step a0, a1;
  typename Share<T, BKM, false, M>::Step b0, b1;
  if (full > 0) {
    a.load(a0, k0);
    b.load(b0, k0);
  }
  // the k that fill no step come first
  if (k0 + full * kK < end) {
    a.load_tail(a1, k0 + full * kK);
    b.load_tail(b1, k0 + full * kK);
    a.store(a1, lds);
    b.store(b1, lds + kTwo);
    __syncthreads();
    step64<T, M>(acc, lds, lds + kTwo);
    __syncthreads();
  }
  if (full == 0) return;
  // no load in these loops is under a condition, so that a wait for the older ones does not wait for the newer
  if constexpr (kSlots<T, M> == 1) {
    for (int s = 1; s < full; ++s) {
      a.store(a0, lds);
      b.store(b0, lds + kTwo);
      a.load(a0, k0 + s * kK);
      b.load(b0, k0 + s * kK);
      __syncthreads();
      step64<T, M>(acc, lds, lds + kTwo);
      __syncthreads();
    }
    a.store(a0, lds);
    b.store(b0, lds + kTwo);
    __syncthreads();
    step64<T, M>(acc, lds, lds + kTwo);
  } else {
    if (full > 1) {
      a.load(a1, k0 + kK);
      b.load(b1, k0 + kK);
    }
    a.store(a0, lds);
    b.store(b0, lds + kTwo);
    int s = 0;
    for (; s + 3 < full; s += 2) {
      a.load(a0, k0 + (s + 2) * kK);
      b.load(b0, k0 + (s + 2) * kK);
      __syncthreads();                       // slot 0 is written, slot 1 has been read
      step64<T, M>(acc, lds, lds + kTwo);
      a.store(a1, lds + 2 * kTwo);
      b.store(b1, lds + 3 * kTwo);
      a.load(a1, k0 + (s + 3) * kK);
      b.load(b1, k0 + (s + 3) * kK);
      __syncthreads();
      step64<T, M>(acc, lds + 2 * kTwo, lds + 3 * kTwo);
      a.store(a0, lds);
      b.store(b0, lds + kTwo);
    }
    // one to three steps are left: s in slot 0, s + 1 on its way
    if (s + 2 < full) {
      a.load(a0, k0 + (s + 2) * kK);
      b.load(b0, k0 + (s + 2) * kK);
    }
    __syncthreads();
    step64<T, M>(acc, lds, lds + kTwo);
    if (s + 1 >= full) return;
    a.store(a1, lds + 2 * kTwo);
    b.store(b1, lds + 3 * kTwo);
    __syncthreads();
    step64<T, M>(acc, lds + 2 * kTwo, lds + 3 * kTwo);
    if (s + 2 >= full) return;
    a.store(a0, lds);
    b.store(b0, lds + kTwo);
    __syncthreads();
    step64<T, M>(acc, lds, lds + kTwo);
  }
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
  __shared__ __attribute__((aligned(16))) T lds[2 * kSlots<T, M> * kSlot<T, M>];
  int mt, nt;
  if (!tile_of(blockIdx.x, tm, tn, mt, nt)) return;
  const int v0 = mt * M, t0 = nt * M;
  constexpr int B = kB<M>;
  int target[B];
#pragma unroll
  for (int j = 0; j < B; ++j) target[j] = t0 + col_of<M>(j) < C ? y[t0 + col_of<M>(j)] - v0 : -1;
  AccM<M> acc;
  tile64<T, false, false, false, M>(acc, Side<T>{W, d, V, d, nullptr}, v0, Side<T>{H, d, C, d, nullptr}, t0, 0, d, lds);
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

// TOKENS a block, 256 / TOKENS threads each.  lse is M + log sum; lp comes from its parts, so that it does not
// carry the rounding of an lse that is much larger, and rest is what that rounding left.
template <int TOKENS>
__global__ void __launch_bounds__(256)
    k64_merge(const float* __restrict__ part_m, const float* __restrict__ part_s,
              const float* __restrict__ zy, const int32_t* __restrict__ y, int V, int tiles,
              int64_t stride, int C, float* __restrict__ lp, float* __restrict__ lse, float* __restrict__ rest) {
  constexpr int kPer = 256 / TOKENS;
  __shared__ float sm[kPer][TOKENS + 1];
  const int c = threadIdx.x % TOKENS, q = threadIdx.x / TOKENS, t = blockIdx.x * TOKENS + c;
  const int at = min(t, C - 1);
  float m = -__builtin_huge_valf();
#pragma unroll 8
  for (int i = q; i < tiles; i += kPer) m = __builtin_elementwise_maximum(m, part_m[i * stride + at]);
  sm[q][c] = m;
  __syncthreads();
#pragma unroll 16
  for (int k = 0; k < kPer; ++k) m = __builtin_elementwise_maximum(m, sm[k][c]);
  float s = 0.f;
#pragma unroll 4
  for (int i = q; i < tiles; i += kPer) {
    const float p = part_s[i * stride + at], pm = part_m[i * stride + at];
    s += p != 0.f ? p * expf(pm - m) : 0.f;
  }
  __syncthreads();
  sm[q][c] = s;
  __syncthreads();
  if (q != 0 || t >= C) return;
  s = 0.f;
#pragma unroll 16
  for (int k = 0; k < kPer; ++k) s += sm[k][c];
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
  __shared__ __attribute__((aligned(16))) T lds[2 * kSlots<T, M> * kSlot<T, M>];
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
    tile64<T, false, false, false, M>(acc, Side<T>{W, d, V, d, nullptr}, v0, Side<T>{H, d, C, d, nullptr}, t0, 0, d, lds);
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

// Four elements of dW.
__device__ __forceinline__ void write_dw(void* dW, int64_t at, f4 x, int accumulate, int bf16) {
  if (bf16) {
    typename Four<__bf16>::type q;
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = (__bf16)x[e];
    *(typename Four<__bf16>::type*)((__bf16*)dW + at) = q;
  } else {
    typedef typename Four<float>::type V4;
    V4* to = (V4*)((float*)dW + at);
    *to = accumulate ? *to + (V4)x : (V4)x;
  }
}

// Workgroups [h_from, h_from + h_grid): dH; [w_from, ...): dW.  Each in shares of its k (share_v of the
// vocabulary, share_c tokens), of which more than one leave their sums in parts.
struct GradSplit {
  int h_from, h_grid, h_shares, share_v;
  int w_from, w_shares, share_c;
  float *h_parts, *w_parts;
  int accumulate, dw_bf16;
};
template <typename T, int M>
__global__ void __launch_bounds__(kThreads64, M == 64 ? 4 : 3)     // (without: 888 us)
    k64_grads(const T* __restrict__ W, const T* __restrict__ H, const T* __restrict__ dZ,
              const float* __restrict__ grad_lp, int V, int d, int C, int vpad, GradSplit p,
              T* __restrict__ dH, void* __restrict__ dW) {
  __shared__ __attribute__((aligned(16))) T lds[2 * kSlots<T, M> * kSlot<T, M>];
  constexpr int B = kB<M>;
  const int tm = (d + M - 1) / M;
  int mt, nt;
  AccM<M> acc;
  if ((unsigned)((int)blockIdx.x - p.h_from) < (unsigned)p.h_grid) {
    const int tn = (C + M - 1) / M;
    // the shares outermost: those of one are on one XCD and read the same rows of W
    if (!tile_of(blockIdx.x - p.h_from, tm, tn * p.h_shares, mt, nt)) return;
    const int share = nt / tn, n0 = mt * M, t0 = (nt - share * tn) * M;
    const int k0 = share * p.share_v, k1 = min(k0 + p.share_v, vpad);
    tile64<T, true, false, false, M>(acc, Side<T>{W, d, d, V, nullptr}, n0, Side<T>{dZ, vpad, C, vpad, nullptr}, t0, k0, k1, lds);
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
        if (p.h_shares > 1) {
          *(f4*)(p.h_parts + ((int64_t)share * C + t) * d + n) = acc[i][j];
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
  const int tn = (V + M - 1) / M;
  if (!tile_of(blockIdx.x - p.w_from, tm, tn * p.w_shares, mt, nt)) return;
  const int share = nt / tn, n0 = mt * M, v0 = (nt - share * tn) * M;
  const int k0 = share * p.share_c, k1 = min(k0 + p.share_c, C);
  tile64<T, true, true, true, M>(acc, Side<T>{H, d, d, C, grad_lp}, n0, Side<T>{dZ, vpad, vpad, C, nullptr}, v0, k0, k1, lds);
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int v = v0 + col_of<M>(j);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int n = n0 + row_of<M>(i);
      if (v >= V || n >= d) continue;
      if (p.w_shares > 1) *(f4*)(p.w_parts + ((int64_t)share * V + v) * d + n) = acc[i][j];
      else write_dw(dW, (int64_t)v * d + n, acc[i][j], p.accumulate, p.dw_bf16);
    }
  }
}

__device__ __forceinline__ f4 sum_of(const float* parts, int64_t n, int shares, int64_t at) {
  f4 s = *(const f4*)(parts + at);
  for (int k = 1; k < shares; ++k) s += *(const f4*)(parts + k * n + at);
  return s;
}

// dH and dW as the sums of their shares, 4 elements a lane: workgroups [0, h_grid) dH.
template <typename T>
__global__ void __launch_bounds__(256)
    k64_join(GradSplit p, int h_grid, int64_t h_n, int64_t w_n, T* __restrict__ dH, void* __restrict__ dW) {
  const bool h = (int)blockIdx.x < h_grid;
  const int64_t at = ((int64_t)((int)blockIdx.x - (h ? 0 : h_grid)) * 256 + threadIdx.x) * 4;
  if (at >= (h ? h_n : w_n)) return;
  if (!h) {
    write_dw(dW, at, sum_of(p.w_parts, w_n, p.w_shares, at), p.accumulate, p.dw_bf16);
    return;
  }
  const f4 s = sum_of(p.h_parts, h_n, p.h_shares, at);
  typename Four<T>::type q;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = (T)s[e];
  *(typename Four<T>::type*)(dH + at) = q;
}

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

// 32 where 64 x 64 tiles would not give every CU one, or tokens (cols) would leave a quarter or more of
// theirs empty that 32 would not.  us, 64 against 32:
//   float32 forward              N = 3       64         300        3000
//   d 64,   V 1000               9    8      10   8     10   9     14   17
//   d 1024, V 64                 29   13     30   13    31   14    31   14
//   d 1024, V 8000               32   17     33   24    65   64
//   d 4096, V 1000               95   33     97   34    98   51
//   d 1024, V 32000              52   38     55   61
//   bfloat16 backward, d 4096, V 1000
//                                33   26     36   29    53   50
//                      d 1024, V 1000
//                                19   16     21   17    23   21    81   87
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
  // more threads a token where its tiles are many and blocks of 16 would leave CUs idle.  us of the
  // forward at d 64, 16 against 4: 16 tokens, V 8000 15 and 11, V 128000 121 and 48; 512 tokens, V 8000
  // 22 and 17; but 2048 tokens, V 1024 12.0 and 13.2; 8192 tokens, V 32000 502 and 540
  const int per = tiles >= 96 && C < 4096 ? 4 : 16;
  const auto k = per == 16 ? k64_merge<16> : k64_merge<4>;
  k<<<cdiv(C, per), 256, 0, s>>>(part_m, part_s, zy, y, (int)V, tiles, stride, C, lp, lse, rest);
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

// Rows and columns of the gradients' tiles: 32 where dW, even in shares, has few of them.
static int grads_rows(int64_t V, int64_t d, int64_t C) {
  return (int64_t)cdiv(d, 64) * cdiv(V, 64) * std::max<int64_t>(1, C / 512) <= 128 ? 32 : 64;
}

// Shares of the tokens that dW's sums are split into, of 8 steps at least, until 512 workgroups share them.
// us of the backward, whole and in shares (and in 64 x 64 tiles, where there are many), float32: 2000 tokens,
// d 64, V 1000 46 and 31; 8000 tokens, d 256, V 1000 336 and 229 (142); 4000, d 512, V 300 159 and 93 (68);
// 7000, d 3328, V 2 260 and 134 (107); 2000, d 256, V 1000 69 in shares of 32 x 32 tiles and 50 in those of 64.
// 1024 workgroups, or 4 steps, take as long or longer (512 tokens, d 256, V 1024: 25 of 8 steps, 27 of 4).
int64_t dw_shares(int64_t V, int64_t d, int64_t C) {
  const int M = grads_rows(V, d, C);
  const int64_t tiles = (int64_t)cdiv(d, M) * cdiv(V, M);
  return std::max<int64_t>(1, std::min<int64_t>(cdiv(512, tiles), C / 512));
}

template <typename T>
hipError_t launch64_grads(const T* W, const T* H, const T* dZ, const float* grad_lp, int64_t V,
                          int64_t d, int C, int64_t vpad, int shares, T* dH, float* parts,
                          float* w_parts, int accumulate, int dw_bf16, void* dW, hipStream_t s) {
  const int M = grads_rows(V, d, C), tm = cdiv(d, M);
  const int w_per = cdiv(cdiv(C, kK), dw_shares(V, d, C));   // steps of a share: none is empty
  GradSplit p{};
  p.h_shares = shares;
  p.share_v = cdiv(vpad / kK, shares) * kK;
  p.w_shares = cdiv(cdiv(C, kK), w_per);
  p.share_c = w_per * kK;
  p.h_parts = parts;
  p.w_parts = w_parts;
  p.accumulate = accumulate;
  p.dw_bf16 = dw_bf16;
  p.h_grid = dH != nullptr ? (int)tile_grid((int64_t)tm * cdiv(C, M) * shares) : 0;
  const int64_t w = dW != nullptr ? tile_grid((int64_t)tm * cdiv(V, M) * p.w_shares) : 0;
  // those with the longer sums first
  if (p.share_c > p.share_v) p.h_from = (int)w;
  else p.w_from = p.h_grid;
  {
    ScopedKernelTimer timer(KK_GRADS64, s);
    const auto k = M == 32 ? k64_grads<T, 32> : k64_grads<T, 64>;
    k<<<(unsigned)(p.h_grid + w), kThreads64, 0, s>>>(W, H, dZ, grad_lp, (int)V, (int)d, C, (int)vpad, p, dH, dW);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t h_n = (int64_t)C * d, w_n = V * d;
  const int h_join = dH != nullptr && p.h_shares > 1 ? cdiv(h_n, 1024) : 0;
  const int w_join = dW != nullptr && p.w_shares > 1 ? cdiv(w_n, 1024) : 0;
  if (h_join + w_join == 0) return hipSuccess;
  ScopedKernelTimer timer(KK_JOIN64, s);
  k64_join<T><<<h_join + w_join, 256, 0, s>>>(p, h_join, h_n, w_n, dH, dW);
  return hipGetLastError();
}

#define GRPO_INSTANTIATE64(T)                                                                     \
  template hipError_t launch64_dz<T>(const T*, const T*, const int32_t*, const float*,            \
                                     const float*, const float*, const float*, int64_t, int64_t,  \
                                     int, int64_t, const LogitXform&, T*, hipStream_t);           \
  template hipError_t launch64_grads<T>(const T*, const T*, const T*, const float*, int64_t,      \
                                        int64_t, int, int64_t, int, T*, float*, float*, int, int, \
                                        void*, hipStream_t);
GRPO_INSTANTIATE64(float)
GRPO_INSTANTIATE64(__bf16)

}  // namespace grpo
