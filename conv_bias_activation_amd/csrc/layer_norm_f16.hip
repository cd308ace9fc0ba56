// layer_norm_f16.hip — layer norm and its gradient, X in f16.
#include "layer_norm.hpp"

namespace biasact {
int launch_layer_norm_f16(int dty, const NormArgs& a, hipStream_t s) { return launch_layer_norm<DT_F16>(dty, a, s); }
int launch_layer_norm_grad_f16(int dty, const NormGradArgs& a, hipStream_t s) { return launch_layer_norm_grad<DT_F16>(dty, a, s); }
}  // namespace biasact
