// The matrix product of the decoder-block operators, f32 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_f32(bool gated, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch<LORA_F32>(gated, shape, a, st);
}

}  // namespace lora
