// The matrix product of the decoder-block operators, bf16 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_bf16(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return gemm::launch_any<LORA_BF16>(form, shape, a, st);
}

int32_t gemm_launch_pair_bf16(int shape, const GemmArgs& x, const GemmArgs& w, hipStream_t st) {
  return gemm::launch_pair<LORA_BF16>(shape, x, w, st);
}

}  // namespace lora
