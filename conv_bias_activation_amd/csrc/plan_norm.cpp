// plan_norm.cpp — argument checking of layer norm, its gradient and the gradient
// of the bias-and-activation epilogue.  Plain C++: no HIP call happens here, so
// every error path is reachable on a machine without a GPU.
#include "norm_plan.hpp"
#include "plan.hpp"

namespace biasact {

namespace {

constexpr int kF32 = 0, kF16 = 1, kBF16 = 2;
constexpr int64_t kMaxBytes = (int64_t)1 << 31;   // every tensor < 2 GiB

int elem_bytes(int dt) { return dt == kF32 ? 4 : 2; }
bool valid_float_dt(int dt) { return dt == kF32 || dt == kF16 || dt == kBF16; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool too_large(int64_t a, int64_t b) { return a > 0 && b >= (kMaxBytes + a - 1) / a; }

// The types and sizes that both layer norm calls check alike.
int norm_common(int64_t rows, int64_t N, uint32_t dtypes, NormPlan* p) {
  if (!p || rows < 0 || N < 0) return kErrInvalid;
  p->dtx = (int)(dtypes & 0xffu);
  p->dtw = (int)((dtypes >> 8) & 0xffu);
  p->dty = (int)((dtypes >> 24) & 0xffu);
  if (!valid_float_dt(p->dtx) || !valid_float_dt(p->dtw) || !valid_float_dt(p->dty) || ((dtypes >> 16) & 0xffu)) return kErrUnsupported;
  const int es = elem_bytes(p->dtx) > elem_bytes(p->dty) ? elem_bytes(p->dtx) : elem_bytes(p->dty);
  if (rows >= kMaxBytes || N >= kMaxBytes || too_large(rows * es, N)) return kErrUnsupported;
  if (too_large(N, elem_bytes(p->dtw)) || too_large(rows, 4)) return kErrUnsupported;   // weights, statistics
  p->empty = rows == 0 || N == 0;
  p->rows = (uint32_t)rows;
  p->N = (uint32_t)N;
  return kOk;
}

bool bad(const void* p, int dt) { return p && !aligned(p, (uintptr_t)elem_bytes(dt)); }

}  // namespace

int plan_layer_norm(const void* X, const void* gamma, const void* beta, const void* Y, const void* mean,
                    const void* rstd, int64_t rows, int64_t N, float eps, uint32_t dtypes, NormPlan* p) {
  const int rc = norm_common(rows, N, dtypes, p);
  if (rc) return rc;
  if (!(eps >= 0.0f) || eps > 3.4028235e38f) return kErrInvalid;
  if (p->empty) return kOk;
  if (!X || !Y || bad(X, p->dtx) || bad(Y, p->dty) || bad(gamma, p->dtw) || bad(beta, p->dtw)) return kErrInvalid;
  if (X == Y && p->dtx != p->dty) return kErrInvalid;  // in place only where the types are equal
  if (!mean != !rstd || bad(mean, kF32) || bad(rstd, kF32)) return kErrInvalid;
  return kOk;
}

size_t layer_norm_grad_workspace(int64_t rows, int64_t N) {
  if (rows <= 0 || N <= 0 || rows >= kMaxBytes || N >= kMaxBytes) return 0;
  // (16-bit types have the most parts)
  return (size_t)norm_grad_parts((uint32_t)rows, (uint32_t)N, 4u) * 2u * (size_t)N * 4u;
}

int plan_layer_norm_grad(const void* dY, const void* X, const void* gamma, const void* mean, const void* rstd,
                         const void* dX, const void* dgamma, const void* dbeta, int64_t rows, int64_t N,
                         uint32_t dtypes, const void* workspace, size_t workspace_bytes, NormPlan* p) {
  const int rc = norm_common(rows, N, dtypes, p);
  if (rc) return rc;
  if (N == 0) return kOk;
  if (bad(dgamma, p->dtw) || bad(dbeta, p->dtw)) return kErrInvalid;
  if (rows == 0) return kOk;
  if (!dY || !X || !mean || !rstd || !dX || bad(dY, p->dty) || bad(X, p->dtx) || bad(dX, p->dtx) || bad(gamma, p->dtw) ||
      bad(mean, kF32) || bad(rstd, kF32))
    return kErrInvalid;
  // in place only where the types are equal, and where no later kernel reads X and dY again
  const bool in_place = dX == X || dX == dY;
  if ((dX == dY && p->dtx != p->dty) || (in_place && N > (int64_t)kNormLong)) return kErrInvalid;
  if ((dgamma || dbeta) &&
      (!workspace || !aligned(workspace, 16) || workspace_bytes < layer_norm_grad_workspace(rows, N)))
    return kErrInvalid;
  return kOk;
}

size_t bias_act_grad_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || M >= kMaxBytes || N >= kMaxBytes) return 0;
  return (size_t)act_grad_parts((uint32_t)M, (uint32_t)N) * (size_t)N * 4u;
}

int plan_bias_act_grad(const void* dY, const void* Z, const void* dZ, const void* dbias, int64_t M, int64_t N,
                       uint32_t dtypes, int act, const void* workspace, size_t workspace_bytes, ActGradPlan* p) {
  if (!p || M < 0 || N < 0 || act < 0 || act > 5) return kErrInvalid;
  p->dt = (int)(dtypes & 0xffu);
  p->dtb = (int)((dtypes >> 16) & 0xffu);
  if (!valid_float_dt(p->dt) || !valid_float_dt(p->dtb) || ((dtypes >> 8) & 0xffu) || (dtypes >> 24)) return kErrUnsupported;
  if (M >= kMaxBytes || N >= kMaxBytes || too_large(M * elem_bytes(p->dt), N)) return kErrUnsupported;
  if (dbias && too_large(N, elem_bytes(p->dtb))) return kErrUnsupported;
  p->M = (uint32_t)M;
  p->N = (uint32_t)N;
  p->empty = M == 0 || N == 0;
  if (N == 0) return kOk;
  if (bad(dbias, p->dtb) || (!dZ && !dbias)) return kErrInvalid;
  if (M == 0) return kOk;
  if (!dY || (!Z && act != 0) || bad(dY, p->dt) || bad(Z, p->dt) || bad(dZ, p->dt)) return kErrInvalid;
  if (dbias && (!workspace || !aligned(workspace, 16) || workspace_bytes < bias_act_grad_workspace(M, N))) return kErrInvalid;
  return kOk;
}

}  // namespace biasact
