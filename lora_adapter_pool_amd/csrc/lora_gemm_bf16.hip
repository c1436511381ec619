// The matrix product of the decoder-block operators, bf16 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_bf16(bool gated, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch<LORA_BF16>(gated, shape, a, st);
}

}  // namespace lora
