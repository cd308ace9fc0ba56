// gemm_mx_bf16.hip — fused product with an MXFP4 B + bias + activation, A in bf16.
#include "gemm_mx_launch.hpp"

namespace biasact {
int launch_gemm_mx_bf16(int dto, const MxGemmArgs& a, hipStream_t s) {
  return launch_gemm_mx<DT_BF16>(dto, a, s);
}
}  // namespace biasact
