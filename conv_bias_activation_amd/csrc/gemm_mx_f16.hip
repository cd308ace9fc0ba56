// gemm_mx_f16.hip — fused product with an MXFP4 B + bias + activation, A in f16.
#include "gemm_mx_launch.hpp"

namespace biasact {
int launch_gemm_mx_f16(int dto, const MxGemmArgs& a, hipStream_t s) {
  return launch_gemm_mx<DT_F16>(dto, a, s);
}
}  // namespace biasact
