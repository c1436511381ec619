// Shared declarations of the decoder-block operators (norm, linear, gated
// feed-forward and its gradients): argument structs of the launchers and the
// device helpers that their epilogues share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "lora_internal.h"

namespace lora {

// One product z[m][n] = sum_k A[m][k] B[n][k] and what its epilogue does.
//   linear: out[m][n] = act(sa[m] sb[n] z + bias[n] + delta[m][n]) + residual[m][n]
//   gated:  B has 2 n rows (gate rows, then up rows); pre = sa sb z + delta,
//           out[m][n] = act(pre[m][n]) * pre[m][n + N]
// A and B are stored with the reduction contiguous; in the gradients' products
// (epilogue as linear) they are stored reduction-major: B as [k][n] in the
// gradient of x, A as [k][m] and B as [k][n] in the gradient of w.
enum Form { kLinearForm = 0, kGatedForm = 1, kGradX = 2, kGradW = 3 };

struct GemmArgs {
  const char* A;
  const char* B;
  const float* sa;        // one scale a row of A, or nullptr
  const float* sb;        // one scale a row of B, or nullptr
  const void* bias;       // [N], or nullptr
  const void* delta;      // [M][N] ([M][2 N] gated), or nullptr
  const void* residual;   // [M][N], or nullptr
  void* pre;              // gated: [M][2 N], or nullptr
  void* out;              // [M][N]
  float* part;            // split K: [tiles - whole][splits][bm][bn] raw products
  int64_t kb;             // bytes of the reduction
  int64_t lda, ldb;       // bytes from a stored row to the next (multiples of 16)
  int32_t M, N;
  int32_t whole;          // tiles that are not split: the first ones
  int32_t splits;         // parts of each other tile
  int32_t lines;          // load whole cache lines where rows do not start at one
  int32_t out_dtype;      // of bias, delta, residual, pre and out
  int32_t act;
  int32_t tiles_m, tiles_n;
};

// Reduction bytes that a tile step takes: 128 (64 bf16, 128 e4m3, 32 fp32),
// one whole cache line of every row.
constexpr int kStepBytes = 128;

// Launch plan of a product: tile shape and K split, from sizes and types alone.
struct GemmPlan {
  int32_t shape;   // index of a tile shape
  int32_t whole;   // tiles that are not split
  int32_t splits;  // parts of each of the others
  int64_t ws_bytes;  // fp32 partials
  float us;        // estimate
};
GemmPlan gemm_plan(int32_t dtype, int32_t out_dtype, Form form, int64_t M, int64_t N,
                   int64_t kb);
int32_t gemm_run(int32_t dtype, Form form, const GemmPlan& plan, GemmArgs a, void* ws,
                 hipStream_t st);
// the shapes that the gradients' products may share a launch with: the ring's
constexpr int kPairShapes = 3;
// per type (each in its own source file)
int32_t gemm_launch_bf16(Form form, int shape, const GemmArgs& a, hipStream_t st);
int32_t gemm_launch_e4m3(Form form, int shape, const GemmArgs& a, hipStream_t st);
int32_t gemm_launch_f32(Form form, int shape, const GemmArgs& a, hipStream_t st);
int32_t gemm_launch_pair_bf16(int shape, const GemmArgs& x, const GemmArgs& w, hipStream_t st);
int32_t gemm_launch_pair_f32(int shape, const GemmArgs& x, const GemmArgs& w, hipStream_t st);

struct TileShape {
  int bm, bn;  // rows of A and rows of B a workgroup covers
};
// shapes, smallest first: three of gemm_ring_kernel, then gemm_phase_kernel's
constexpr int kNumShapes = 4;
constexpr TileShape kShapes[kNumShapes] = {{32, 32}, {64, 64}, {128, 128}, {256, 256}};
// and gemm_rows_kernel, for few rows, and its waves
constexpr int kRowsShape = kNumShapes, kMostRows = 32, kRowsWaves = 8;

int32_t check_launch(const char* what);
int32_t check_rows(int32_t T);

#ifdef __HIPCC__

typedef uint32_t bk_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t bk_u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float bk_f32x4 __attribute__((ext_vector_type(4)));
typedef float bk_f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float bk_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bk_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bk_bf16x8 __attribute__((ext_vector_type(8)));
typedef int bk_i32x8 __attribute__((ext_vector_type(8)));

// two fp32 -> packed bf16, nearest, ties to even
__device__ __forceinline__ uint32_t bk_pack(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(bk_f32x2{lo, hi}, bk_bf16x2));
}
__device__ __forceinline__ float bk_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bk_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// e^z.  The hardware's exponential is base 2; the product z log2(e) is kept
// with the part that its rounding loses, or the result's relative error would
// grow with |z| (2^-24 |z| log2 e).
__device__ __forceinline__ float bk_exp(float z) {
  constexpr float kL = 1.44269504088896341f, kLlo = 1.92596299e-8f;
  const float p = z * kL;
  const float r = __builtin_fmaf(z, kLlo, __builtin_fmaf(z, kL, -p));
  const float e = __builtin_amdgcn_exp2f(p);
  // From p = 128 on e is infinite, and with a residual of zero or below the
  // correction would make a NaN of it: e alone is right there (a logistic of 0).
  return __builtin_fabsf(p) < 128.f ? __builtin_fmaf(e, r * 0.693147180559945309f, e) : e;
}
// 1 / (1 + e^-z)
__device__ __forceinline__ float bk_logistic(float z) {
  return __builtin_amdgcn_rcpf(1.f + bk_exp(-z));
}
// gelu in its tanh form: 0.5 (1 + tanh u) = logistic(2 u)
constexpr float kGeluC = 0.797884560802865356f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
// the normal distribution's cumulative function; through erfc, which keeps
// its relative accuracy for negative z
__device__ __forceinline__ float bk_phi(float z) {
  return 0.5f * erfcf(-0.707106781186547524f * z);
}
// The same for results that are rounded to bf16: without the correction of the
// exponent (2^-17 of the result at |z| = 100, half a step of bf16 is 2^-9).
// Activations are a large tile's epilogue: 65536 of them on one compute unit.
__device__ __forceinline__ float bk_logistic_short(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
}
// Phi by the Chebyshev fit of erfc in "Numerical Recipes" (erfcc): t e^(-x^2 +
// P(t)), t = 1 / (1 + x / 2), to 1.2e-7 of the result for x >= 0 (and 2^-23 x^2
// of it for the rounding of x^2); no branches.
__device__ __forceinline__ float bk_phi_short(float z) {
  const float x = __builtin_fabsf(0.707106781186547524f * z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.f));
  float q = 0.17087277f;
  q = __builtin_fmaf(q, t, -0.82215223f);
  q = __builtin_fmaf(q, t, 1.48851587f);
  q = __builtin_fmaf(q, t, -1.13520398f);
  q = __builtin_fmaf(q, t, 0.27886807f);
  q = __builtin_fmaf(q, t, -0.18628806f);
  q = __builtin_fmaf(q, t, 0.09678418f);
  q = __builtin_fmaf(q, t, 0.37409196f);
  q = __builtin_fmaf(q, t, 1.00002368f);
  q = __builtin_fmaf(q, t, __builtin_fmaf(-x, x, -1.26551223f));
  const float half = 0.5f * t * __builtin_amdgcn_exp2f(1.44269504088896341f * q);
  return z < 0.f ? half : 1.f - half;  // (a NaN is one in `half`)
}

// Applies an activation to eight values; kShort: for results in bf16.  z = -inf
// would give -inf 0: the factor below is finite, and 0 times it is 0.
template <bool kShort, int NV>
__device__ __forceinline__ void act_apply(int act, float (&z)[NV]) {
  constexpr float kLowest = -0x1.fffffep127f;
  if (act == LORA_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      z[i] = fmaxf(z[i], kLowest) * (kShort ? bk_logistic_short(z[i]) : bk_logistic(z[i]));
  } else if (act == LORA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      z[i] = fmaxf(z[i], kLowest) * (kShort ? bk_phi_short(z[i]) : bk_phi(z[i]));
  } else if (act == LORA_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float v = 2.f * kGeluC * __builtin_fmaf(kGeluA * z[i] * z[i], z[i], z[i]);
      z[i] = fmaxf(z[i], kLowest) * (kShort ? bk_logistic_short(v) : bk_logistic(v));
    }
  } else if (act == LORA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];  // keeps NaN
  }
}

// An activation's value and derivative.  Past the clamps every factor beside
// z is 0 or 1 in fp32, and infinities get the curve's limits: 0 below, z and 1
// above.  (A NaN reaches the result through p.)
template <bool kShort>
__device__ __forceinline__ void act_curve(int act, float z, float& value, float& slope) {
  value = z;
  slope = 1.f;
  const float low = fmaxf(z, -0x1.fffffep127f);
  const float near = fminf(fmaxf(z, -200.f), 200.f);
  if (act == LORA_ACT_SILU) {
    const float p = kShort ? bk_logistic_short(z) : bk_logistic(z);
    value = low * p;
    slope = p * __builtin_fmaf(near, 1.f - p, 1.f);
  } else if (act == LORA_ACT_GELU) {
    const float p = kShort ? bk_phi_short(z) : bk_phi(z);
    const float e = kShort ? __builtin_amdgcn_exp2f(-0.5f * 1.44269504088896341f * near * near)
                           : bk_exp(-0.5f * near * near);
    value = low * p;
    slope = __builtin_fmaf(near * 0.398942280401432678f, e, p);
  } else if (act == LORA_ACT_GELU_TANH) {
    const float v = 2.f * kGeluC * __builtin_fmaf(kGeluA * z * z, z, z);
    const float p = kShort ? bk_logistic_short(v) : bk_logistic(v);
    value = low * p;
    slope = __builtin_fmaf(near * p * (1.f - p),
                           2.f * kGeluC * __builtin_fmaf(3.f * kGeluA * near, near, 1.f), p);
  } else if (act == LORA_ACT_RELU) {
    value = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : z < 0.f ? 0.f : z;  // 0 at 0; keeps NaN
  }
}

// Eight consecutive elements of a row of bf16 or fp32 at element `i`, as far
// as `left` (>= 1) goes; rows of odd length start at any element, and global
// memory takes 16-byte accesses at any element's alignment.
__device__ __forceinline__ void load8(const void* base, int64_t i, int left, int dtype,
                                      float (&v)[8]) {
  if (dtype == LORA_BF16) {
    const uint16_t* p = (const uint16_t*)base + i;
    if (left >= 8) {
      const bk_u32x4 w = *reinterpret_cast<const bk_u32x4_a2*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = bk_lo(w[j]), v[2 * j + 1] = bk_hi(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? __uint_as_float((uint32_t)p[j] << 16) : 0.f;
    }
  } else {
    const float* p = (const float*)base + i;
    if (left >= 8) {
      const bk_f32x4 a = *reinterpret_cast<const bk_f32x4_a4*>(p);
      const bk_f32x4 b = *reinterpret_cast<const bk_f32x4_a4*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.f;
    }
  }
}
__device__ __forceinline__ void store8(void* base, int64_t i, int left, int dtype,
                                       const float (&v)[8]) {
  if (dtype == LORA_BF16) {
    uint16_t* p = (uint16_t*)base + i;
    bk_u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bk_pack(v[2 * j], v[2 * j + 1]);
    if (left >= 8) {
      *reinterpret_cast<bk_u32x4_a2*>(p) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  } else {
    float* p = (float*)base + i;
    if (left >= 8) {
      *reinterpret_cast<bk_f32x4_a4*>(p) = bk_f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<bk_f32x4_a4*>(p + 4) = bk_f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) p[j] = v[j];
    }
  }
}

// What an epilogue reads beside the products, for eight columns of a row: it
// is fetched for several rows before the first of them is finished, so that
// one latency is waited for and not one a row.  bf16 outputs only (a fetch of
// fp32 would take twice the registers).
template <bool kGated>
struct Extra {
  bk_u32x4 d[kGated ? 2 : 1], r;
};

__device__ __forceinline__ bk_u32x4 load8_raw(const void* base, int64_t i, int left) {
  const uint16_t* p = (const uint16_t*)base + i;
  if (left >= 8) return *reinterpret_cast<const bk_u32x4_a2*>(p);
  bk_u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  return w;
}

template <bool kGated>
__device__ __forceinline__ void fetch_extra(const GemmArgs& p, int m, int n, Extra<kGated>& x) {
  if (m >= p.M || n >= p.N) return;
  const int left = p.N - n;
  if constexpr (kGated) {
    const int64_t at = (int64_t)m * 2 * p.N + n;
    if (p.delta) {
      x.d[0] = load8_raw(p.delta, at, left);
      x.d[1] = load8_raw(p.delta, at + p.N, left);
    }
  } else {
    const int64_t at = (int64_t)m * p.N + n;
    if (p.delta) x.d[0] = load8_raw(p.delta, at, left);
    if (p.residual) x.r = load8_raw(p.residual, at, left);
  }
}

__device__ __forceinline__ void add8(float (&z)[8], const bk_u32x4& w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) z[2 * j] += bk_lo(w[j]), z[2 * j + 1] += bk_hi(w[j]);
}
__device__ __forceinline__ void add8(float (&z)[8], const void* base, int64_t i, int left,
                                     int dtype) {
  float t[8];
  load8(base, i, left, dtype, t);
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] += t[j];
}

// The epilogue on eight raw products of row m, columns n .. n + 8 (n < N);
// kFetched: bf16 outputs, delta and residual already in `x`.
template <bool kGated, bool kFetched>
__device__ __forceinline__ void epilogue8(const GemmArgs& p, int m, int n, float (&z)[8],
                                          float (&u)[8], const Extra<kGated>& x) {
  const int left = p.N - n;
  const int od = kFetched ? (int)LORA_BF16 : p.out_dtype;
  if (p.sa) {
    float t[8];
    const float s = p.sa[m];
    load8(p.sb, n, left, LORA_F32, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = z[j] * s * t[j];
    if constexpr (kGated) {
      load8(p.sb, (int64_t)p.N + n, left, LORA_F32, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = u[j] * s * t[j];
    }
  }
  if constexpr (kGated) {
    const int64_t at = (int64_t)m * 2 * p.N + n;
    if (p.delta) {
      if constexpr (kFetched) {
        add8(z, x.d[0]);
        add8(u, x.d[1]);
      } else {
        add8(z, p.delta, at, left, od);
        add8(u, p.delta, at + p.N, left, od);
      }
    }
    if (p.pre) {
      store8(p.pre, at, left, od, z);
      store8(p.pre, at + p.N, left, od, u);
    }
    if (od == LORA_BF16)
      act_apply<true>(p.act, z);
    else
      act_apply<false>(p.act, z);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] *= u[j];
    store8(p.out, (int64_t)m * p.N + n, left, od, z);
  } else {
    const int64_t at = (int64_t)m * p.N + n;
    if (p.bias) add8(z, p.bias, n, left, od);
    if (p.delta) {
      if constexpr (kFetched)
        add8(z, x.d[0]);
      else
        add8(z, p.delta, at, left, od);
    }
    if (od == LORA_BF16)
      act_apply<true>(p.act, z);
    else
      act_apply<false>(p.act, z);
    if (p.residual) {
      if constexpr (kFetched)
        add8(z, x.r);
      else
        add8(z, p.residual, at, left, od);
    }
    store8(p.out, at, left, od, z);
  }
}

// Workgroup -> XCD: workgroups are dealt round-robin to the 8 XCDs, each with
// an L2 of its own; XCD x takes the x-th contiguous eighth of `total` items.
__device__ __forceinline__ int xcd_item(int b, int total) {
  const int q = total >> 3, r = total & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}
// Tiles go in groups of 8 row tiles, columns outside, so that the workgroups
// that run together share rows of A and of B.
__device__ __forceinline__ void tile_place(const GemmArgs& p, int id, int& tm, int& tn) {
  const int gsz = 8 * p.tiles_n, g = id / gsz, first = 8 * g;
  const int rows = p.tiles_m - first < 8 ? p.tiles_m - first : 8;
  id -= g * gsz;
  tm = first + id % rows;
  tn = id / rows;
}

#endif  // __HIPCC__

}  // namespace lora
