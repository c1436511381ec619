// The matrix product of the decoder-block operators, f32 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_f32(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch_any<LORA_F32>(form, shape, a, st);
}

int32_t gemm_launch_pair_f32(int shape, const GemmArgs& x, const GemmArgs& w, hipStream_t st) {
  return gemm::launch_pair<LORA_F32>(shape, x, w, st);
}

}  // namespace lora
