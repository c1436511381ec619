// The matrix product of the decoder-block operators, f32 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_f32(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch_any<LORA_F32>(form, shape, a, st);
}

}  // namespace lora
