// gemm_mx_mxfp4.hip — fused product with an MXFP4 B + bias + activation, A in mxfp4.
#include "gemm_mx_launch.hpp"

namespace biasact {
int launch_gemm_mx_mxfp4(int dto, const MxGemmArgs& a, hipStream_t s) {
  return launch_gemm_mx<DT_MXFP4>(dto, a, s);
}
}  // namespace biasact
