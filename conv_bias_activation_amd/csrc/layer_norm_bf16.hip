// layer_norm_bf16.hip — layer norm and its gradient, X in bf16.
#include "layer_norm.hpp"

namespace biasact {
int launch_layer_norm_bf16(int dty, const NormArgs& a, hipStream_t s) { return launch_layer_norm<DT_BF16>(dty, a, s); }
int launch_layer_norm_grad_bf16(int dty, const NormGradArgs& a, hipStream_t s) { return launch_layer_norm_grad<DT_BF16>(dty, a, s); }
}  // namespace biasact
