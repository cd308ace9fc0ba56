// gemm_f8_wide_bf16.hip — fused product of two 8-bit operands + bias + activation, bf16 output, sums in fp32.
#include "gemm_f8.hpp"

namespace biasact {
void launch_gemm_f8_wide_bf16(const F8GemmArgs& a, hipStream_t s) { launch_gemm_f8<DT_BF16, true>(a, s); }
}  // namespace biasact
