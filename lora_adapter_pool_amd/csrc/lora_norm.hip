// Root-mean-square norm with the residual's addition and an output in 8 bits.
//
//   t = round(x + residual)                      (the stream the next layer reads)
//   n = t * (mean(t^2) + eps)^(-1/2) * weight
//   out = round(n);  scale = max(max |n| / 448, 2^-126);  out8 = e4m3(n r),
//   r = 1 / scale rounded to fp32
//
// One pass over memory: a row stays in registers (up to four pieces of eight
// elements a thread) between the statistic and the outputs, so the bytes are
// x and the residual once in, every output once out.  The row's statistic
// is summed in 64 bits: the rounding of n r to 8 bits has borders, and a
// statistic that is right to 32 bits leaves n with the three roundings of its
// products alone.  (n r differs from n / scale in its last bits, so from e4m3 of
// the quotient only at such a border.)  The workgroup size is the row's, because a row's latency
// (load, two reductions, store) is what a small batch waits for; large batches
// run at the rate of a copy (8960 x 4096 bf16 with residual and 8-bit output:
// 330 MB in 61 us, 5.4 TB/s).
#include <hip/hip_runtime.h>

#include "lora_block.h"

namespace lora {

namespace {

constexpr int kMaxPieces = 4;
constexpr int kMaxThreads = 1024;
constexpr int kMaxHidden = kMaxThreads * kMaxPieces * 8;

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum;
  void* out;
  uint8_t* out8;
  float* scale;
  int32_t H;
  double over_h, eps;
};

// 1 / x and 1 / sqrt(x) to within a few steps of 64 bits: the hardware's
// estimates (some 2^-26) and one step of third order.  Zero and infinity keep
// the estimate's infinity and zero.
__device__ __forceinline__ double reciprocal(double x) {
  const double y = __builtin_amdgcn_rcp(x), e = __builtin_fma(-x, y, 1.0);
  const double z = __builtin_fma(y, __builtin_fma(e, e, e), y);
  return e == e ? z : y;
}
__device__ __forceinline__ double reciprocal_root(double x) {
  const double y = __builtin_amdgcn_rsq(x), e = __builtin_fma(-x * y, y, 1.0);
  const double z = __builtin_fma(y, e * __builtin_fma(0.375, e, 0.5), y);
  return e == e ? z : y;
}

// A piece of eight elements as it is stored (the weights are fetched with the
// row, and take their room before its statistic is known).
template <int DT>
struct Raw {
  bk_u32x4 v[DT == LORA_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const bk_u32x4* p = reinterpret_cast<const bk_u32x4*>(
        (const char*)base + i * (DT == LORA_F32 ? 4 : 2));
    v[0] = p[0];
    if constexpr (DT == LORA_F32) v[1] = p[1];
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == LORA_F32) return __uint_as_float(v[i >> 2][i & 3]);
    const uint32_t w = v[0][i >> 1];
    return i & 1 ? bk_hi(w) : bk_lo(w);
  }
};

// NP pieces of eight elements a thread, one row a workgroup.
template <int DT, int NP>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a) {
  __shared__ double sums[kMaxThreads / 64];
  __shared__ uint32_t tops[kMaxThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x, waves = nt >> 6;
  const int64_t base = (int64_t)blockIdx.x * a.H;
  float t[NP][8];
  Raw<DT> weight[NP];
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
      load8(a.x, base + c, 8, DT, t[j]);
      weight[j].load(a.weight, c);
      if (a.residual) {
        float r[8];
        load8(a.residual, base + c, 8, DT, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[j][i] += r[i];
        if constexpr (DT == LORA_BF16) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint32_t w = bk_pack(t[j][i], t[j][i + 1]);
            t[j][i] = bk_lo(w);
            t[j][i + 1] = bk_hi(w);
          }
        }
        store8(a.sum, base + c, 8, DT, t[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)t[j][i], (double)t[j][i], ss);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = 0.f;
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) ss += __shfl_xor(ss, d);
  if (waves > 1) {
    if ((tid & 63) == 0) sums[tid >> 6] = ss;
    __syncthreads();
    ss = 0.0;
    for (int i = 0; i < waves; ++i) ss += sums[i];  // same order in every thread
  }
  const double root = reciprocal_root(__builtin_fma(ss, a.over_h, a.eps));
  float rstd = (float)root;
  // A row of numbers below 2^-128, or near the largest, has a factor that fp32
  // does not hold, or not with all its bits: part of it goes to the row first.
  if (root > 0x1p120 || root < 0x1p-120) {
    const float part = root > 1.0 ? 0x1p64f : 0x1p-64f;
    rstd = (float)(root * (root > 1.0 ? 0x1p-64 : 0x1p64));
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] *= part;
  }

  uint32_t top = 0;  // largest |n| by its bits, which also keeps a NaN
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = (tid + j * nt) * 8;
    if (c < a.H) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[j][i] = t[j][i] * rstd * weight[j].at(i);
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

template <int DT>
void launch_norm(const NormArgs& a, int T, hipStream_t st) {
  const int pieces = a.H / 8;
  // One piece a thread up to 512 threads (64 rows of 4096: 3.7 us against 4.3
  // with two, 8960 rows 61 against 64), then two (8960 rows of 8192 bf16: 68 us
  // against 95 with 1024 threads of one), then 1024 threads.
  int nt = 64;
  while (nt < 512 && nt < pieces) nt *= 2;
  if (nt * 2 < pieces) nt = kMaxThreads;
  const int np = (pieces + nt - 1) / nt;
  if (np == 1)
    hipLaunchKernelGGL((norm_kernel<DT, 1>), dim3(T), dim3(nt), 0, st, a);
  else if (np == 2)
    hipLaunchKernelGGL((norm_kernel<DT, 2>), dim3(T), dim3(nt), 0, st, a);
  else
    hipLaunchKernelGGL((norm_kernel<DT, kMaxPieces>), dim3(T), dim3(nt), 0, st, a);
}

}  // namespace

}  // namespace lora

extern "C" int32_t lora_add_rms_norm(const lora_norm_desc* desc, const void* x,
                                     const void* residual, const void* weight, void* sum,
                                     void* out, void* out8, float* scale, int32_t T,
                                     void* stream) {
  using namespace lora;
  clear_error();
  if (!desc) return fail(LORA_E_ARG, "descriptor is NULL");
  if (desc->dtype != LORA_F32 && desc->dtype != LORA_BF16)
    return fail(LORA_E_DTYPE, "norm dtype must be fp32 or bf16, got %d", desc->dtype);
  if (desc->hidden < 8 || desc->hidden > kMaxHidden)
    return fail(LORA_E_SHAPE, "hidden must be in [8, %d], got %d", kMaxHidden, desc->hidden);
  if (desc->hidden % 8)
    return fail(LORA_E_ALIGN, "hidden must be a multiple of 8, got %d", desc->hidden);
  if (!(desc->eps >= 0.f && desc->eps < __builtin_inff()))
    return fail(LORA_E_ARG, "eps must be finite and >= 0, got %g", (double)desc->eps);
  if (int32_t e = check_rows(T)) return e;
  if (T == 0) return LORA_OK;
  if (!x || !weight) return fail(LORA_E_ARG, "x and weight must not be NULL");
  if ((residual != nullptr) != (sum != nullptr))
    return fail(LORA_E_ARG, "residual and sum go together: one of them is NULL");
  if ((out8 != nullptr) != (scale != nullptr))
    return fail(LORA_E_ARG, "out8 and scale go together: one of them is NULL");
  if (!out && !out8) return fail(LORA_E_ARG, "out and out8 are both NULL");
  const void* ptrs[] = {x, residual, weight, sum, out, out8, scale};
  for (const void* p : ptrs)
    if (!aligned16(p))
      return fail(LORA_E_ALIGN, "every buffer of the norm must be 16-byte aligned");
  const NormArgs a{x,     residual, weight, sum, out, (uint8_t*)out8,
                   scale, desc->hidden, 1.0 / desc->hidden, (double)desc->eps};
  if (desc->dtype == LORA_BF16)
    launch_norm<LORA_BF16>(a, T, (hipStream_t)stream);
  else
    launch_norm<LORA_F32>(a, T, (hipStream_t)stream);
  return check_launch("norm");
}
