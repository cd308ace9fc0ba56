// gemm_f8_f32.hip — fused product of two 8-bit operands + bias + activation, f32 output.
#include "gemm_f8.hpp"

namespace biasact {
void launch_gemm_f8_f32(const F8GemmArgs& a, hipStream_t s) { launch_gemm_f8<DT_F32, true>(a, s); }
}  // namespace biasact
