// layer_norm_f32.hip — layer norm and its gradient, X in f32.
#include "layer_norm.hpp"

namespace biasact {
int launch_layer_norm_f32(int dty, const NormArgs& a, hipStream_t s) { return launch_layer_norm<DT_F32>(dty, a, s); }
int launch_layer_norm_grad_f32(int dty, const NormGradArgs& a, hipStream_t s) { return launch_layer_norm_grad<DT_F32>(dty, a, s); }
}  // namespace biasact
