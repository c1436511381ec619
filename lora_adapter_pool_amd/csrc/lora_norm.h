// Device helpers that the norms share.
#pragma once

#include "lora_block.h"

#ifdef __HIPCC__

namespace lora {

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
  // from a uniform address and an offset in bytes
  __device__ __forceinline__ void load_at(const void* base, uint32_t at) {
    const bk_u32x4* p = reinterpret_cast<const bk_u32x4*>((const char*)base + at);
    v[0] = p[0];
    if constexpr (DT == LORA_F32) v[1] = p[1];
  }
  // What was unpacked or computed from the piece before is not kept for what follows.
  __device__ __forceinline__ void opaque() {
#pragma unroll
    for (bk_u32x4& p : v) asm volatile("" : "+v"(p));
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == LORA_F32) return __uint_as_float(v[i >> 2][i & 3]);
    const uint32_t w = v[0][i >> 1];
    return i & 1 ? bk_hi(w) : bk_lo(w);
  }
};

}  // namespace lora

#endif  // __HIPCC__
