// The matrix product of the decoder-block operators, bf16 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_bf16(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch_any<LORA_BF16>(form, shape, a, st);
}

}  // namespace lora
