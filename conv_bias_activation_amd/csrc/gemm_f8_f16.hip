// gemm_f8_f16.hip — fused product of two 8-bit operands + bias + activation, f16 output.
#include "gemm_f8.hpp"

namespace biasact {
void launch_gemm_f8_f16(const F8GemmArgs& a, hipStream_t s) { launch_gemm_f8<DT_F16, false>(a, s); }
}  // namespace biasact
