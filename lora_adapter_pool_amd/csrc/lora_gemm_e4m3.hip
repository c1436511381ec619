// The matrix product of the decoder-block operators, e4m3 operands.
#include "lora_gemm.h"

namespace lora {

int32_t gemm_launch_e4m3(Form form, int shape, const GemmArgs& a, hipStream_t st) {
  return a.out_dtype == LORA_F32 ? gemm::launch<gemm::kE4m3Exact>(form, shape, a, st)
                                 : gemm::launch<LORA_E4M3>(form, shape, a, st);
}

}  // namespace lora
