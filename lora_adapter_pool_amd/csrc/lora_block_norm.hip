// What joins a block's output to the residual stream and opens the next block,
// and its gradients.
//
//   p = y (mean(y^2) + eps)^(-1/2) post_weight          (p = y without one)
//   t = round(alpha residual + beta gate p)             (the stream)
//   n = t (mean(t^2) + eps)^(-1/2) pre_weight, out = round(n), out8 and scale
//       as lora_add_rms_norm's
//
// One pass over memory: a row stays in registers between the two statistics.
// The row's second statistic depends on its first, so a row waits for two
// reductions over the workgroup; with several rows a compute unit in flight the
// loads of the others fill that time.
//
// Backwards, with a hat for the normalised rows (t_hat = t r_t, r_t the root's
// reciprocal) and < > for a row's mean:
//   dt = dsum + r_t (dout w_pre - t_hat <dout w_pre t_hat>)
//   dresidual = alpha dt,  dgate = beta dt p,  dp = beta gate dt
//   dy = r_y (dp w_post - y_hat <dp w_post y_hat>)
//   dw_pre = sum_rows dout t_hat,  dw_post = sum_rows dp y_hat, and dgate's sum
//   over the rows where the gate is one a channel
// The statistics are made again from y and the stream, which have to be read
// anyhow, so that the forward pass keeps nothing else, and in 64 bits as there: a
// row's factors are the same numbers in both passes, and rows of any size take the same
// path (squares summed in fp32 where they fit, and such rows of zeros again: 108 us for
// the case below, not 112, and 163 where half of the rows are zeros, not 112).  A workgroup takes every
// n-th row and keeps the columns' sums in registers; their partials are added in
// a second launch, in an order that depends on the sizes alone.
//
// Measured (us, bf16): 8960 x 4096 with an element gate and 8-bit output 72, 5.6 TB/s;
// its gradients with a channel gate 112, 3.9 TB/s (a row waits for two reductions, and
// vector units issue in 47% of the cycles), 5 of it the sums' launch.  64 rows 4.2 to
// 4.7, a launch's time.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lora_norm.h"

namespace lora {

namespace {

constexpr int kMaxHidden = 16384;
constexpr int kForwardThreads = 1024, kBackwardThreads = 512;
// Workgroups that keep sums over rows: as many as a compute unit holds at once, two of 256
// or 512 threads, one of 512 with more than one piece a thread (8960 x 8192 bf16 222 us,
// with two in turn 234), more where they are smaller (8960 x 1024 39 us, with two 60), but
// four rows each (700 x 1024 12 us, with a row each 14: every one writes its sums).
inline int sum_groups(int H, int T) {
  int n = H > 4096 ? 256 : 512;
  for (int h = 2048; h >= H && n < 4096; h /= 2) n *= 2;
  if (n > 512) n = std::min(n, std::max(T / 4, 512));
  return std::min(n, T);
}

struct JoinArgs {
  const void* y;
  const void* residual;
  const void* gate;
  const void* post;
  const void* pre;
  void* sum;
  void* out;
  uint8_t* out8;
  float* scale;
  int64_t gate_row;  // elements from a row's gate to the next: H, or 0
  int32_t H;
  float alpha, beta;
  double over_h, eps;
};

// A statistic's factor, in two parts: fp32 does not hold the factor of a row of
// numbers below 2^-128, or near the largest, or not with all its bits.
struct Factor {
  float part, rest;
  __device__ __forceinline__ void times(float (&x)[8]) const {
    if (part != 1.f)  // (the same for the whole row)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= part;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= rest;
  }
};
__device__ __forceinline__ Factor factor_of(double root) {
  if (root > 0x1p120) return {0x1p64f, (float)(root * 0x1p-64)};
  if (root < 0x1p-120) return {0x1p-64f, (float)(root * 0x1p64)};
  return {1.f, (float)root};
}

// A value of another lane of the same 16, by a lane move (no trip through LDS); all
// lanes of the wave have to be active.
template <int kMove>
__device__ __forceinline__ double moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, kMove, 15, 15, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), kMove, 15, 15, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// Sums over 16 lanes, the same in each (a tree whose branches commute).
template <int N>
__device__ __forceinline__ void sum_over_16(double (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += moved<kXor1>(v[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += moved<kXor2>(v[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += moved<kHalfMirror>(v[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += moved<kMirror>(v[k]);
}
// Sums over the workgroup, the same in every thread.  `room` (a place for each of up to
// 16 waves) is not read again before another barrier has passed.
template <int N>
__device__ __forceinline__ void sum_over(double (&v)[N], double (*room)[N]) {
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  sum_over_16(v);
#pragma unroll
  for (int d = 16; d < 64; d *= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], d);
  if (waves == 1) return;
  if ((tid & 63) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) room[tid >> 6][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const double w = room[tid & 15][k];  // (past the last wave: not written, and not taken)
    v[k] = (tid & 15) < waves ? w : 0.0;
  }
  sum_over_16(v);
}

__device__ __forceinline__ double square_plus(float x, double s) {
  return __builtin_fma((double)x, (double)x, s);
}

template <int DT, int NP>
__global__ __launch_bounds__(kForwardThreads) void join_kernel(JoinArgs a) {
  __shared__ double first[16][1], second[16][1];
  __shared__ uint32_t tops[kForwardThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x, waves = nt >> 6;
  const int64_t base = (int64_t)blockIdx.x * a.H, gate = blockIdx.x * a.gate_row;
  float t[NP][8];
  Raw<DT> residual[NP], post[NP], pre[NP], g[NP];
  double ss[1] = {0.0};
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
      load8(a.y, base + c, 8, DT, t[j]);
      residual[j].load(a.residual, base + c);
      if (a.post) post[j].load(a.post, c);
      if (a.gate) g[j].load(a.gate, gate + c);
      if (a.pre) pre[j].load(a.pre, c);
      if (a.post)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = square_plus(t[j][i], ss[0]);
    }
  }
  if (a.post) {
    sum_over(ss, first);
    const Factor f = factor_of(reciprocal_root(__builtin_fma(ss[0], a.over_h, a.eps)));
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      f.times(t[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] *= post[j].at(i);
    }
  }
  ss[0] = 0.0;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.gate) t[j][i] *= g[j].at(i);
        t[j][i] = residual[j].at(i) * a.alpha + t[j][i] * a.beta;
      }
      if constexpr (DT == LORA_BF16) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t w = bk_pack(t[j][i], t[j][i + 1]);
          t[j][i] = bk_lo(w);
          t[j][i + 1] = bk_hi(w);
        }
      }
      store8(a.sum, base + c, 8, DT, t[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = square_plus(t[j][i], ss[0]);
    }
  }
  if (!a.pre) return;
  sum_over(ss, second);
  const Factor f = factor_of(reciprocal_root(__builtin_fma(ss[0], a.over_h, a.eps)));
  uint32_t top = 0;  // largest |n| by its bits, which also keeps a NaN
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
      f.times(t[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[j][i] *= pre[j].at(i);
        const uint32_t b = __float_as_uint(t[j][i]) & 0x7fffffffu;
        top = b > top ? b : top;
      }
      if (a.out) store8(a.out, base + c, 8, DT, t[j]);
    }
  }
  if (!a.out8) return;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  if (waves > 1) {
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    for (int i = 0; i < waves; ++i) top = tops[i] > top ? tops[i] : top;
  }
  float scale = (float)((double)__uint_as_float(top) * (1.0 / 448.0));
  scale = scale < 0x1p-126f ? 0x1p-126f : scale;  // keeps NaN
  const float inv = (float)reciprocal(scale);
  if (tid == 0) a.scale[blockIdx.x] = scale;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[j][0] * inv, t[j][1] * inv, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[j][2] * inv, t[j][3] * inv, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[j][4] * inv, t[j][5] * inv, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[j][6] * inv, t[j][7] * inv, hi, true);
      *reinterpret_cast<uint64_t*>(a.out8 + base + c) =
          (uint32_t)lo | (uint64_t)(uint32_t)hi << 32;
    }
  }
}

// The row's threads: one piece of eight elements a thread up to `most`.
inline int threads_of(int H, int most) {
  int nt = 64;
  while (nt < most && nt < H / 8) nt *= 2;
  return nt;
}

template <int DT>
void launch_join(const JoinArgs& a, int T, hipStream_t st) {
  const int nt = threads_of(a.H, 512) * (a.H > 8192 ? 2 : 1);
  if (a.H / 8 <= nt)
    hipLaunchKernelGGL((join_kernel<DT, 1>), dim3(T), dim3(nt), 0, st, a);
  else
    hipLaunchKernelGGL((join_kernel<DT, 2>), dim3(T), dim3(nt), 0, st, a);
}

struct BackArgs {
  const void* dout;
  const void* dsum;
  const void* y;
  const void* sum;
  const void* gate;
  const void* post;
  const void* pre;
  void* dy;
  void* dresidual;
  void* dgate;   // [T][H], or nullptr
  float* part;   // [kinds][workgroups][H]: sums over a workgroup's rows
  int32_t k_pre, k_post, k_gate;  // which kind each sum is, or -1
  int64_t gate_row;
  int32_t H, T;
  float alpha, beta;
  double over_h, eps;
};

// Sum of eight products in fp32, in three levels: off by at most four half steps of the
// sum of their magnitudes.  For the products with the normalised y, which are of dp's
// size; sums of squares, and of products with the stream itself, are of any size.
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __builtin_fmaf(a[2 * i], b[2 * i], a[2 * i + 1] * b[2 * i + 1]);
  return (p[0] + p[1]) + (p[2] + p[3]);
}

// Eight elements to a uniform address and an offset in bytes.
template <int DT>
__device__ __forceinline__ void put8(void* base, uint32_t at, const float (&v)[8]) {
  bk_u32x4* p = reinterpret_cast<bk_u32x4*>((char*)base + at);
  if constexpr (DT == LORA_BF16) {
    *p = bk_u32x4{bk_pack(v[0], v[1]), bk_pack(v[2], v[3]), bk_pack(v[4], v[5]),
                  bk_pack(v[6], v[7])};
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      p[h] = bk_u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                      __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
  }
}

// A thread's pieces of a row, as they are stored.
template <int DT, int N>
struct BackRow {
  Raw<DT> y[N], t[N], dout[N], dsum[N], gate[N];
};

// The parts that a call has are the kernel's (kPre: a norm before the next block,
// kPost: one after this, kGate), not questions at every element (8960 x 4096 bf16: 132
// us with them).
template <int DT, int NP, bool kPre, bool kPost, bool kGate>
__global__ __launch_bounds__(kBackwardThreads, DT == LORA_BF16 && NP == 1 ? 4 : 2)
void join_backward_kernel(BackArgs a) {
  // One piece a thread, or two of bf16: the next row's are fetched while this one is worked
  // on.  Four pieces leave no registers to hold a row over the reductions: it is read
  // again, from the caches.
  constexpr bool kAhead = NP == 1 || (NP == 2 && DT == LORA_BF16);
  constexpr uint32_t ES = DT == LORA_F32 ? 4 : 2;
  constexpr int kHeld = NP < 4 ? NP : 1;
  // by the row's parity: a row's reductions may meet the next row's writes
  __shared__ double first[2][16][3], second[2][16][1];
  const int tid = threadIdx.x, nt = blockDim.x;
  float w_pre[NP][8] = {}, w_post[NP][8] = {}, w_gate[NP][8] = {};  // sums over the rows
  Raw<DT> pre[kHeld], post[kHeld];
  BackRow<DT, kHeld> now, next;
  // (a row's address is uniform: one offset of 32 bits serves all arrays)
  auto at_row = [&](const void* p, int64_t row) {
    return (const void*)((const char*)p + row * ES);
  };
  // what the first reduction does not take
  auto load_rest = [&](int row, int j, uint32_t c, BackRow<DT, kHeld>& r) {
    if (a.dsum) r.dsum[j % kHeld].load_at(at_row(a.dsum, (int64_t)row * a.H), c * ES);
    if (kGate) r.gate[j % kHeld].load_at(at_row(a.gate, row * a.gate_row), c * ES);
  };
  auto load_row = [&](int row, int j, uint32_t c, BackRow<DT, kHeld>& r) {
    const int64_t base = (int64_t)row * a.H;
    const int k = j % kHeld;
    if (kPost || kGate) r.y[k].load_at(at_row(a.y, base), c * ES);
    if (kPre) {
      r.t[k].load_at(at_row(a.sum, base), c * ES);
      r.dout[k].load_at(at_row(a.dout, base), c * ES);
    }
    if constexpr (!kAhead) load_rest(row, j, c, r);
  };
  auto load_weights = [&](int j, uint32_t c) {
    if (kPre) pre[j % kHeld].load_at(a.pre, c * ES);
    if (kPost) post[j % kHeld].load_at(a.post, c * ES);
  };
  if (kAhead)
#pragma unroll
    for (int j = 0; j < NP; ++j)
      if ((tid + j * nt) * 8 < a.H) load_row(blockIdx.x, j, (tid + j * nt) * 8, next);
  int parity = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, parity ^= 1) {
    const int64_t base = (int64_t)row * a.H;
    // (sums of the arrays' addresses and the thread's place are not kept over the rows)
    uint32_t mine = (uint32_t)tid * 8;
    if constexpr (kAhead) {
      asm volatile("" : "+v"(mine));
      now = next;
      const int after = row + (int)gridDim.x;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const uint32_t c = mine + (uint32_t)(j * nt) * 8;
        if (c < (uint32_t)a.H) {
          load_rest(row, j, c, now);
          if (after < a.T) load_row(after, j, c, next);
        }
      }
    }
    double s[3] = {0.0, 0.0, 0.0};  // of t^2, dout w_pre t and y^2
    // (One piece a thread, four waves a SIMD: elements are unpacked again behind the
    // reduction, and y's behind t's; kept over them they are more than the registers.)
    auto stat = [&](int j) {
      const int k = j % kHeld;
      if (kPre) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double x = now.t[k].at(i);
          s[0] = __builtin_fma(x, x, s[0]);
          s[1] = __builtin_fma((double)(now.dout[k].at(i) * pre[k].at(i)), x, s[1]);
        }
        if (NP == 1) now.t[k].opaque(), now.dout[k].opaque(), pre[k].opaque();
      }
      if (kPost) {
        if (NP == 1 && kPre) now.y[k].opaque();
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] = square_plus(now.y[k].at(i), s[2]);
        if (NP == 1) now.y[k].opaque();
      }
    };
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const uint32_t c = mine + (uint32_t)(j * nt) * 8;
      if (c < (uint32_t)a.H) {
        if constexpr (!kAhead) load_row(row, j, c, now);
        load_weights(j, c);
        if constexpr (kHeld < NP) stat(j);
      }
    }
    if constexpr (kHeld == NP)
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (mine + (uint32_t)(j * nt) * 8 < (uint32_t)a.H) stat(j);
    if (kPre || kPost) sum_over(s, first[parity]);
    const double rt = reciprocal_root(__builtin_fma(s[0], a.over_h, a.eps));
    const double ry = reciprocal_root(__builtin_fma(s[2], a.over_h, a.eps));
    const Factor ft = factor_of(rt), fy = factor_of(ry);
    const float ct = (float)(s[1] * rt * a.over_h);
    float dp[NP][8];
    double s2[1] = {0.0};
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const uint32_t c = mine + (uint32_t)(j * nt) * 8, k = j % kHeld;
      if (c < (uint32_t)a.H) {
        if constexpr (kHeld < NP) {
          __builtin_amdgcn_sched_barrier(0);  // (a piece's loads and no more at a time)
          load_row(row, j, c, now);
          load_weights(j, c);
        }
        float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, z[8];
        if (kPre) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = now.t[k].at(i);
          ft.times(z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = now.dout[k].at(i);
            w_pre[j][i] = __builtin_fmaf(o, z[i], w_pre[j][i]);
            d[i] = __builtin_fmaf(-z[i], ct, o * pre[k].at(i));
          }
          ft.times(d);
        }
        if (a.dsum)
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += now.dsum[k].at(i);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = a.alpha * d[i];
        if (a.dresidual) put8<DT>((void*)at_row(a.dresidual, base), c * ES, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] *= a.beta;
          z[i] = kPost || kGate ? now.y[k].at(i) : 0.f;
        }
        if (kPost) fy.times(z);
        if (kGate) {
          float dg[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dg[i] = d[i] * (kPost ? z[i] * post[k].at(i) : z[i]);
            w_gate[j][i] += dg[i];
            d[i] *= now.gate[k].at(i);
          }
          if (a.dgate) put8<DT>((void*)at_row(a.dgate, base), c * ES, dg);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (kPost) {
            w_post[j][i] = __builtin_fmaf(d[i], z[i], w_post[j][i]);
            d[i] *= post[k].at(i);
          }
          dp[j][i] = d[i];
        }
        // (with y normalised: the product with y itself may be past fp32's range)
        if (kPost) s2[0] += (double)dot8(dp[j], z);
        if (!kPost && a.dy) put8<DT>((void*)at_row(a.dy, base), c * ES, dp[j]);
      }
    }
    if (kPost && a.dy) {
      sum_over(s2, second[parity]);
      const float cy = (float)(s2[0] * a.over_h);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const uint32_t c = mine + (uint32_t)(j * nt) * 8, k = j % kHeld;
        if (c < (uint32_t)a.H) {
          float d[8];
          if constexpr (kHeld < NP) now.y[k].load_at(at_row(a.y, base), c * ES);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = now.y[k].at(i);
          fy.times(d);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = __builtin_fmaf(-d[i], cy, dp[j][i]);
          fy.times(d);
          put8<DT>((void*)at_row(a.dy, base), c * ES, d);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const uint32_t c = (uint32_t)(tid + j * nt) * 8;
    if (c < (uint32_t)a.H) {
      const int64_t n = gridDim.x, at = (int64_t)blockIdx.x * a.H + c;
      if (kPre && a.k_pre >= 0) store8(a.part, a.k_pre * n * a.H + at, 8, LORA_F32, w_pre[j]);
      if (kPost && a.k_post >= 0) store8(a.part, a.k_post * n * a.H + at, 8, LORA_F32, w_post[j]);
      if (kGate && a.k_gate >= 0) store8(a.part, a.k_gate * n * a.H + at, 8, LORA_F32, w_gate[j]);
    }
  }
}

// The partials' sums.  A workgroup takes kCols columns of one kind, its threads every
// (1024 / kCols)-th partial.  25 MB of partials for 4096 columns of three kinds: 5.2 us;
// with few columns there are few workgroups, so that they take half as many (8960 x 1024
// in all 38.6 us against 41.0; a quarter 41.7).
struct SumArgs {
  const float* part;
  float* to[3];
  int32_t groups, H, accumulate;
};
template <int kCols>
__global__ __launch_bounds__(1024) void column_sums(SumArgs a) {
  __shared__ float room[16][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = threadIdx.x % kCols, c = blockIdx.x * kCols + col;
  const float* from = a.part + (int64_t)blockIdx.y * a.groups * a.H + c;
  float s = 0.f;
  if (c < a.H)
#pragma unroll 8
    for (int r = threadIdx.x / kCols; r < a.groups; r += 1024 / kCols) s += from[(int64_t)r * a.H];
#pragma unroll
  for (int d = kCols; d < 64; d *= 2) s += __shfl_xor(s, d);
  if (lane < kCols) room[wave][lane] = s;
  __syncthreads();
  if ((int)threadIdx.x >= kCols || c >= a.H) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += room[i][lane];
  float* to = blockIdx.y == 0 ? a.to[0] : blockIdx.y == 1 ? a.to[1] : a.to[2];
  to[c] = a.accumulate ? to[c] + s : s;
}

template <int DT, int NP, bool kPre, bool kPost>
void launch_parts(const BackArgs& a, int groups, int nt, hipStream_t st) {
  if (a.gate)
    hipLaunchKernelGGL((join_backward_kernel<DT, NP, kPre, kPost, true>), dim3(groups), dim3(nt), 0,
                       st, a);
  else
    hipLaunchKernelGGL((join_backward_kernel<DT, NP, kPre, kPost, false>), dim3(groups), dim3(nt),
                       0, st, a);
}
template <int DT, int NP>
void launch_pieces(const BackArgs& a, int groups, int nt, hipStream_t st) {
  if (a.pre)
    a.post ? launch_parts<DT, NP, true, true>(a, groups, nt, st)
           : launch_parts<DT, NP, true, false>(a, groups, nt, st);
  else
    a.post ? launch_parts<DT, NP, false, true>(a, groups, nt, st)
           : launch_parts<DT, NP, false, false>(a, groups, nt, st);
}
template <int DT>
void launch_backward(const BackArgs& a, int groups, hipStream_t st) {
  // Two pieces a thread for rows of more than 2048 columns, where a workgroup has more than
  // a row to go through: a wave's share of the reductions is half (8960 x 4096 bf16 119 ->
  // 112 us, fp32 205 -> 188; 2560 columns 88 -> 86 and 156 -> 127; 700 x 4096 19.9 -> 19.7
  // and 28.2 -> 25.6), and with fewer rows, where more threads wait for a row's loads at
  // once, one (256 x 4096 12.7 against 13.1, fp32 14.3 against 15.1).  By the sizes alone, so
  // that a row's gradients do not depend on which sums are wanted.
  int nt = threads_of(a.H, kBackwardThreads);
  if (nt == kBackwardThreads && a.H / 8 <= nt && a.T > 512) nt /= 2;
  const int np = (a.H / 8 + nt - 1) / nt;
  if (np == 1)
    launch_pieces<DT, 1>(a, groups, nt, st);
  else if (np == 2)
    launch_pieces<DT, 2>(a, groups, nt, st);
  else
    launch_pieces<DT, 4>(a, groups, nt, st);
}

int32_t check_join(const lora_block_norm_desc* d) {
  if (!d) return fail(LORA_E_ARG, "descriptor is NULL");
  if (d->dtype != LORA_F32 && d->dtype != LORA_BF16)
    return fail(LORA_E_DTYPE, "block norm dtype must be fp32 or bf16, got %d", d->dtype);
  if (d->hidden < 8 || d->hidden > kMaxHidden)
    return fail(LORA_E_SHAPE, "hidden must be in [8, %d], got %d", kMaxHidden, d->hidden);
  if (d->hidden % 8)
    return fail(LORA_E_ALIGN, "hidden must be a multiple of 8, got %d", d->hidden);
  if (!(d->eps >= 0.f && d->eps < __builtin_inff()))
    return fail(LORA_E_ARG, "eps must be finite and >= 0, got %g", (double)d->eps);
  if (d->gate < LORA_GATE_NONE || d->gate > LORA_GATE_ELEMENT)
    return fail(LORA_E_ARG, "unknown gate %d", d->gate);
  if (!(__builtin_fabsf(d->residual_scale) < __builtin_inff()) ||
      !(__builtin_fabsf(d->block_scale) < __builtin_inff()))
    return fail(LORA_E_ARG, "the scales of residual and block must be finite");
  return LORA_OK;
}

int32_t check_aligned(const void* const* p, int n) {
  for (int i = 0; i < n; ++i)
    if (!aligned16(p[i]))
      return fail(LORA_E_ALIGN, "every buffer of the block norm must be 16-byte aligned");
  return LORA_OK;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" int32_t lora_block_norm(const lora_block_norm_desc* desc, const void* y,
                                   const void* residual, const void* gate,
                                   const void* post_weight, const void* pre_weight, void* sum,
                                   void* out, void* out8, float* scale, int32_t T,
                                   void* stream) {
  clear_error();
  if (int32_t e = check_join(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return LORA_OK;
  if (!y || !residual || !sum)
    return fail(LORA_E_ARG, "y, residual and sum must not be NULL");
  if ((gate != nullptr) != (desc->gate != LORA_GATE_NONE))
    return fail(LORA_E_ARG, "the gate is NULL, or the descriptor has none");
  if ((out8 != nullptr) != (scale != nullptr))
    return fail(LORA_E_ARG, "out8 and scale go together: one of them is NULL");
  if ((pre_weight != nullptr) != (out || out8))
    return fail(LORA_E_ARG, "pre_weight and an output go together");
  const void* ptrs[] = {y, residual, gate, post_weight, pre_weight, sum, out, out8, scale};
  if (int32_t e = check_aligned(ptrs, 9)) return e;
  const JoinArgs a{y,
                   residual,
                   gate,
                   post_weight,
                   pre_weight,
                   sum,
                   out,
                   (uint8_t*)out8,
                   scale,
                   desc->gate == LORA_GATE_ELEMENT ? desc->hidden : 0,
                   desc->hidden,
                   desc->residual_scale,
                   desc->block_scale,
                   1.0 / desc->hidden,
                   (double)desc->eps};
  if (desc->dtype == LORA_BF16)
    launch_join<LORA_BF16>(a, T, (hipStream_t)stream);
  else
    launch_join<LORA_F32>(a, T, (hipStream_t)stream);
  return check_launch("block norm");
}

extern "C" int64_t lora_block_norm_backward_workspace_bytes(const lora_block_norm_desc* desc,
                                                            int32_t T) {
  clear_error();
  if (int32_t e = check_join(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  return (int64_t)3 * sum_groups(desc->hidden, T) * desc->hidden * 4;
}

extern "C" int32_t lora_block_norm_backward(
    const lora_block_norm_desc* desc, const void* dout, const void* dsum, const void* y,
    const void* sum, const void* gate, const void* post_weight, const void* pre_weight, void* dy,
    void* dresidual, void* dgate, float* dpost_weight, float* dpre_weight, int32_t accumulate,
    int32_t T, void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (int32_t e = check_join(desc)) return e;
  if (int32_t e = check_rows(T)) return e;
  if (accumulate != 0 && accumulate != 1)
    return fail(LORA_E_ARG, "accumulate must be 0 or 1, got %d", accumulate);
  if (dgate && desc->gate == LORA_GATE_NONE)
    return fail(LORA_E_ARG, "dgate, and the descriptor has no gate");
  const bool element = desc->gate == LORA_GATE_ELEMENT;
  if (T) {
    if (dpost_weight && !post_weight)
      return fail(LORA_E_ARG, "dpost_weight without post_weight");
    if (dpre_weight && !pre_weight) return fail(LORA_E_ARG, "dpre_weight without pre_weight");
    if (!dy && !dresidual && !dgate && !dpost_weight && !dpre_weight)
      return fail(LORA_E_ARG, "every output is NULL");
    if ((post_weight || desc->gate != LORA_GATE_NONE) && !y)
      return fail(LORA_E_ARG, "y is NULL, and a norm or a gate takes it");
    if ((gate != nullptr) != (desc->gate != LORA_GATE_NONE))
      return fail(LORA_E_ARG, "the gate is NULL, or the descriptor has none");
    if ((pre_weight != nullptr) != (dout != nullptr))
      return fail(LORA_E_ARG, "pre_weight and dout go together: one of them is NULL");
    if (pre_weight && !sum) return fail(LORA_E_ARG, "pre_weight without the kept sum");
    if (!dout && !dsum) return fail(LORA_E_ARG, "dout and dsum are both NULL");
  }
  const void* ptrs[] = {dout, dsum,      y,     sum,          gate,        post_weight, pre_weight,
                        dy,   dresidual, dgate, dpost_weight, dpre_weight, ws};
  if (int32_t e = check_aligned(ptrs, 13)) return e;
  SumArgs s{};
  BackArgs a{};
  int kinds = 0;
  a.k_pre = a.k_post = a.k_gate = -1;
  if (dpre_weight) s.to[kinds] = dpre_weight, a.k_pre = kinds++;
  if (dpost_weight) s.to[kinds] = dpost_weight, a.k_post = kinds++;
  if (dgate && !element) s.to[kinds] = (float*)dgate, a.k_gate = kinds++;
  // without sums over the rows nothing is kept from row to row
  const int groups = kinds ? sum_groups(desc->hidden, T) : T;
  if (kinds && T) {
    const int64_t need = lora_block_norm_backward_workspace_bytes(desc, T);
    if (!ws) return fail(LORA_E_ARG, "workspace is NULL");
    if (ws_bytes < need)
      return fail(LORA_E_WORKSPACE, "workspace holds %lld bytes, the call needs %lld",
                  (long long)ws_bytes, (long long)need);
  }
  const hipStream_t st = (hipStream_t)stream;
  if (T) {
    a.dout = dout;
    a.dsum = dsum;
    a.y = y;
    a.sum = sum;
    a.gate = gate;
    a.post = post_weight;
    a.pre = pre_weight;
    a.dy = dy;
    a.dresidual = dresidual;
    a.dgate = element ? dgate : nullptr;
    a.part = (float*)ws;
    a.gate_row = element ? desc->hidden : 0;
    a.H = desc->hidden;
    a.T = T;
    a.alpha = desc->residual_scale;
    a.beta = desc->block_scale;
    a.over_h = 1.0 / desc->hidden;
    a.eps = (double)desc->eps;
    if (desc->dtype == LORA_BF16)
      launch_backward<LORA_BF16>(a, groups, st);
    else
      launch_backward<LORA_F32>(a, groups, st);
    if (int32_t e = check_launch("block norm backward")) return e;
  }
  if (!kinds || (!T && accumulate)) return LORA_OK;
  s.part = (const float*)ws;
  s.groups = T ? groups : 0;
  s.H = desc->hidden;
  s.accumulate = accumulate;
  if (desc->hidden > 1024)
    hipLaunchKernelGGL(column_sums<64>, dim3((desc->hidden + 63) / 64, kinds), dim3(1024), 0, st,
                       s);
  else
    hipLaunchKernelGGL(column_sums<32>, dim3((desc->hidden + 31) / 32, kinds), dim3(1024), 0, st,
                       s);
  return check_launch("sums over the rows");
}
