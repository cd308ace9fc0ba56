// api_norm.hip — the extern "C" entry points of layer norm, its gradient and the
// gradient of the bias-and-activation epilogue (include/biasact.h).  Each call
// checks its arguments (plan_norm.cpp), then queues its kernels on the caller's
// stream.  Nothing is allocated or synchronised here.
#include "biasact.h"
#include "launch_kernel.hpp"
#include "norm_args.hpp"
#include "norm_plan.hpp"
#include "plan.hpp"

using namespace biasact;

extern "C" {

int layer_norm(const void* X, const void* gamma, const void* beta, void* Y, float* mean, float* rstd, int64_t rows,
               int64_t N, float eps, uint32_t dtypes, hipStream_t stream) {
  NormPlan p;
  int rc = plan_layer_norm(X, gamma, beta, Y, mean, rstd, rows, N, eps, dtypes, &p);
  if (rc || p.empty) return rc;
  const NormArgs a = {X, gamma, beta, Y, mean, rstd, p.rows, p.N, p.dtw, eps};
  switch (p.dtx) {
    case DT_F32: rc = launch_layer_norm_f32(p.dty, a, stream); break;
    case DT_F16: rc = launch_layer_norm_f16(p.dty, a, stream); break;
    default: rc = launch_layer_norm_bf16(p.dty, a, stream); break;
  }
  return rc ? kErrUnsupported : launch_status();
}

size_t layer_norm_grad_workspace_size(int64_t rows, int64_t N) { return layer_norm_grad_workspace(rows, N); }

int layer_norm_grad(const void* dY, const void* X, const void* gamma, const float* mean, const float* rstd, void* dX,
                    void* dgamma, void* dbeta, int64_t rows, int64_t N, uint32_t dtypes, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  NormPlan p;
  int rc = plan_layer_norm_grad(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, rows, N, dtypes, workspace, workspace_bytes, &p);
  if (rc || p.N == 0) return rc;
  const bool sums = dgamma || dbeta;
  const uint32_t parts = p.rows ? norm_grad_parts(p.rows, p.N, (p.dtx == DT_F32 ? 4u : 2u) + (p.dty == DT_F32 ? 4u : 2u)) : 0u;
  if (p.rows) {
    const NormGradArgs a = {dY, X, gamma, mean, rstd, dX, sums ? static_cast<float*>(workspace) : nullptr, p.rows, p.N, parts, p.dtw};
    switch (p.dtx) {
      case DT_F32: rc = launch_layer_norm_grad_f32(p.dty, a, stream); break;
      case DT_F16: rc = launch_layer_norm_grad_f16(p.dty, a, stream); break;
      default: rc = launch_layer_norm_grad_bf16(p.dty, a, stream); break;
    }
    if (rc) return kErrUnsupported;
  }
  // (without rows: zeros)
  if (sums) launch_join_columns(JoinArgs{static_cast<const float*>(workspace), {dgamma, dbeta}, parts, p.N, 2u * p.N, p.dtw}, stream);
  return launch_status();
}

size_t bias_act_grad_workspace_size(int64_t M, int64_t N) { return bias_act_grad_workspace(M, N); }

int bias_act_grad(const void* dY, const void* Z, void* dZ, void* dbias, int64_t M, int64_t N, uint32_t dtypes, int act,
                  float alpha, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ActGradPlan p;
  const int rc = plan_bias_act_grad(dY, Z, dZ, dbias, M, N, dtypes, act, workspace, workspace_bytes, &p);
  if (rc || p.N == 0) return rc;
  const uint32_t parts = p.M ? act_grad_parts(p.M, p.N) : 0u;
  if (p.M) {
    const ActGradArgs a = {dY, Z, dZ, dbias ? static_cast<float*>(workspace) : nullptr, p.M, p.N, parts, act_grad_lane_bits(p.N), act, alpha};
    if (launch_act_grad(p.dt, a, stream)) return kErrUnsupported;
  }
  if (dbias) launch_join_columns(JoinArgs{static_cast<const float*>(workspace), {dbias, nullptr}, parts, p.N, p.N, p.dtb}, stream);
  return launch_status();
}

}  // extern "C"
