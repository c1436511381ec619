// Gradients of the adapters' delta: geometry shared by the host plan and the
// kernels.
#pragma once

#include "lora_internal.h"

namespace lora {

constexpr int kDeltaTileRows = 64;      // rows of a shrink's or a dx's workgroup
constexpr int kDeltaColumnBytes = 256;  // columns of a gradient's workgroup, in stored bytes
constexpr int kDeltaColumns = 512;      // columns of a dx's workgroup
constexpr int64_t kDeltaAim = 512;      // workgroups wanted, two a compute unit
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

// Bytes of the parts of a workspace: the rows' rank-space values (u of every
// slice, then v of every slice) as the products take them, partials of their
// reductions, partials of the gradients.
struct DeltaLayout {
  int64_t ranks, partial, grads, total;  // byte offsets of the last two, and the end
};
DeltaLayout delta_layout(const Geo& g, int32_t T);

// fp32 values of one slot's gradients (A's, then B's), as a partial holds them
inline int64_t delta_grad_values(const Geo& g) {
  return (int64_t)g.R * ((int64_t)g.S * g.K + g.O);
}

int32_t delta_check_plan(const Geo& g, int32_t T, const lora_delta_plan* p);

}  // namespace lora
