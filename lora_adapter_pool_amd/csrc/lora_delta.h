// Gradients of the adapters' delta: geometry shared by the host plan and the
// kernels.
#pragma once

#include "lora_internal.h"

namespace lora {

constexpr int kDeltaTileRows = 64;      // rows of a shrink's or a dx's workgroup
constexpr int kDeltaColumnBytes = 512;  // columns of a gradient's workgroup, in stored bytes
constexpr int64_t kDeltaAim = 512;      // workgroups of the gradients, two a compute unit
// Workgroups of the ranks, four a compute unit: 53 us and a join of 9.5 for 8704 x 4096 x
// 4096 of 64 ranks; two a unit 56 and 7, reductions never cut 66 (gate/up: 235, and 190 with
// 7 for the join).
constexpr int64_t kDeltaShrinks = 1024;
constexpr int kDeltaMaxSplits = 8;

// Rank tiles of 16 in a rank block, rank blocks, and the ranks they pad to.
struct DeltaRanks {
  int32_t tiles, blocks, padded;
};
inline DeltaRanks delta_ranks(int32_t R) {
  const int32_t t = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  const int32_t b = (R + 16 * t - 1) / (16 * t);
  return {t, b, b * t * 16};
}
inline int32_t delta_column_tile(const Geo& g) {
  return kDeltaColumnBytes / (int32_t)elem_bytes(g.dtype);
}

// A workspace's parts (byte offsets): the rows' rank-space values (u of every slice,
// then v of every slice) ranks outside, u rows outside in fp32, partials of their reductions,
// partials of the gradients.
struct DeltaLayout {
  int64_t turned, straight, partial, grads, total;
};
DeltaLayout delta_layout(const Geo& g, int32_t T);

// fp32 values of one slot's gradients (A's, then B's), as a partial holds them
inline int64_t delta_grad_values(const Geo& g) {
  return (int64_t)g.R * ((int64_t)g.S * g.K + g.O);
}

int32_t delta_check_plan(const Geo& g, int32_t T, const lora_delta_plan* p);

}  // namespace lora
