// plan_mx.cpp — argument checking of the MXFP4 entry points.  Plain C++: no
// HIP call happens here, so every error path is reachable on a machine
// without a GPU.
#include "plan.hpp"

namespace biasact {

namespace {

constexpr int kF32 = 0, kF16 = 1, kBF16 = 2, kMxfp4 = 5;
constexpr int64_t kMaxBytes = (int64_t)1 << 31;   // every tensor < 2 GiB (32-bit buffer offsets)

int elem_bytes(int dt) { return dt == kF32 ? 4 : 2; }
bool valid_float_dt(int dt) { return dt == kF32 || dt == kF16 || dt == kBF16; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
int64_t groups_of(int64_t K) { return (K + 127) / 128; }

// An MXFP4 operand of `rows` rows of G groups: 16-byte aligned codes and
// 4-byte aligned scales (whole words are read and written), each < 2 GiB.
int check_packed(const void* codes, const void* scales, int64_t rows, int64_t G) {
  if (rows > 0 && G > 0) {
    if (rows * G >= kMaxBytes / 64) return kErrUnsupported;
    if (!codes || !scales) return kErrInvalid;
    if (!aligned(codes, 16) || !aligned(scales, 4)) return kErrInvalid;
  }
  return kOk;
}

}  // namespace

int plan_mx_quant(const void* X, const void* codes, const void* scales, int64_t rows, int64_t K, int k_axis,
                  uint32_t dtype, MxQuantPlan* p) {
  if (!p || rows < 0 || K < 0 || (k_axis != 0 && k_axis != 1)) return kErrInvalid;
  if (dtype > 0xffu || !valid_float_dt((int)dtype)) return kErrUnsupported;
  if (rows >= kMaxBytes || K >= kMaxBytes) return kErrUnsupported;
  const int64_t es = elem_bytes((int)dtype);
  if (rows > 0 && K >= (kMaxBytes + rows * es - 1) / (rows * es)) return kErrUnsupported;
  const int64_t G = groups_of(K);
  p->empty = rows == 0 || K == 0;
  if (p->empty) return kOk;
  const int rc = check_packed(codes, scales, rows, G);
  if (rc) return rc;
  if (!X || !aligned(X, (uintptr_t)es)) return kErrInvalid;
  p->dt = (int)dtype;
  p->rows = (uint32_t)rows;
  p->K = (uint32_t)K;
  p->G = (uint32_t)G;
  return kOk;
}

int plan_mx_gemm(const void* A, const void* As, const void* B, const void* Bs, const void* bias, const void* R,
                 const void* C, int64_t M, int64_t N, int64_t K, uint32_t dtypes, int act, MxGemmPlan* p) {
  if (!p || M < 0 || N < 0 || K < 0) return kErrInvalid;
  if (act < 0 || act > 5) return kErrInvalid;
  const int a = (int)(dtypes & 0xffu), b = (int)((dtypes >> 8) & 0xffu);
  const int dtb = (int)((dtypes >> 16) & 0xffu), out = (int)((dtypes >> 24) & 0xffu);
  if (b != kMxfp4 || !(a == kMxfp4 || a == kF16 || a == kBF16)) return kErrUnsupported;
  if (!valid_float_dt(out) || (bias && !valid_float_dt(dtb))) return kErrUnsupported;
  if (a != kMxfp4 && As) return kErrInvalid;             // scales go with an MXFP4 A only
  if (M >= kMaxBytes || N >= kMaxBytes || K >= kMaxBytes) return kErrUnsupported;
  const int64_t G = groups_of(K), so = elem_bytes(out);
  p->empty = M == 0 || N == 0;
  if (p->empty) return kOk;
  if (M >= (kMaxBytes + N * so - 1) / (N * so)) return kErrUnsupported;
  int rc = check_packed(B, Bs, N, G);
  if (rc) return rc;
  if (a == kMxfp4) {
    rc = check_packed(A, As, M, G);
    if (rc) return rc;
  } else if (K > 0) {
    if (M >= (kMaxBytes + 2 * K - 1) / (2 * K)) return kErrUnsupported;
    if (!A || !aligned(A, 2)) return kErrInvalid;
  }
  if (!C || !aligned(C, (uintptr_t)so) || (R && !aligned(R, (uintptr_t)so))) return kErrInvalid;
  if (bias && !aligned(bias, (uintptr_t)elem_bytes(dtb))) return kErrInvalid;
  p->dta = a;
  p->dto = out;
  p->bias_dt = bias ? dtb : -1;
  p->M = (uint32_t)M;
  p->N = (uint32_t)N;
  p->K = (uint32_t)K;
  p->G = (uint32_t)G;
  p->a_bytes = (uint32_t)(a == kMxfp4 ? M * G * 64 : M * K * 2);
  p->as_bytes = (uint32_t)(a == kMxfp4 ? M * G * 4 : 0);
  p->b_bytes = (uint32_t)(N * G * 64);
  p->bs_bytes = (uint32_t)(N * G * 4);
  p->bias_bytes = bias ? (uint32_t)(N * elem_bytes(dtb)) : 0u;
  p->c_bytes = (uint32_t)(M * N * so);
  return kOk;
}

}  // namespace biasact
