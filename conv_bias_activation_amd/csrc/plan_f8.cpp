// plan_f8.cpp — argument checking of the 8-bit floating-point entry points.
// Plain C++: no HIP call happens here, so every error path is reachable on a
// machine without a GPU.
#include "plan.hpp"

namespace biasact {

namespace {

constexpr int kF32 = 0, kF16 = 1, kBF16 = 2, kE4m3 = 6, kE5m2 = 7;
constexpr int kSumsF32 = 0x40;                    // BA_SUMS_F32, beside the output's code
constexpr int64_t kMaxBytes = (int64_t)1 << 31;   // every tensor < 2 GiB (32-bit buffer offsets)

int elem_bytes(int dt) { return dt == kF32 ? 4 : 2; }
bool valid_float_dt(int dt) { return dt == kF32 || dt == kF16 || dt == kBF16; }
bool valid_f8(int dt) { return dt == kE4m3 || dt == kE5m2; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// a * b >= kMaxBytes, for non-negative a and b below it
bool too_large(int64_t a, int64_t b) { return a > 0 && b >= (kMaxBytes + a - 1) / a; }

// An operand's codes (16-byte aligned: whole chunks are moved) and scales
// (4-byte: whole words), each < 2 GiB.
int check_packed(const void* codes, const void* scales, int64_t rows, int64_t K, int block_rows, int64_t* cb,
                 int64_t* sb) {
  const int rc = f8_sizes(rows, K, block_rows, cb, sb);
  if (rc) return rc;
  if (*cb > 0) {
    if (!codes || !scales) return kErrInvalid;
    if (!aligned(codes, 16) || !aligned(scales, 4)) return kErrInvalid;
  }
  return kOk;
}

}  // namespace

int f8_sizes(int64_t rows, int64_t K, int block_rows, int64_t* codes_bytes, int64_t* scales_bytes) {
  if (rows < 0 || K < 0 || !codes_bytes || !scales_bytes || (block_rows != 1 && block_rows != 128)) return kErrInvalid;
  if (rows >= kMaxBytes || K >= kMaxBytes) return kErrUnsupported;
  const int64_t kp = (K + 127) / 128 * 128;
  if (too_large(rows, kp)) return kErrUnsupported;
  *codes_bytes = rows * kp;
  *scales_bytes = (rows + block_rows - 1) / block_rows * ((K + 511) / 512 * 4);
  return kOk;
}

int plan_f8_quant(const void* X, const void* codes, const void* scales, int64_t rows, int64_t K, int k_axis,
                  int block_rows, uint32_t dtypes, F8QuantPlan* p) {
  if (!p || rows < 0 || K < 0 || (k_axis != 0 && k_axis != 1) || (block_rows != 1 && block_rows != 128)) return kErrInvalid;
  const int dt = (int)(dtypes & 0xffu), f8 = (int)((dtypes >> 8) & 0xffu);
  if ((dtypes >> 16) || !valid_float_dt(dt) || !valid_f8(f8)) return kErrUnsupported;
  if (rows >= kMaxBytes || K >= kMaxBytes || too_large(rows * elem_bytes(dt), K)) return kErrUnsupported;
  p->empty = rows == 0 || K == 0;
  if (p->empty) return kOk;
  int64_t cb, sb;
  const int rc = check_packed(codes, scales, rows, K, block_rows, &cb, &sb);
  if (rc) return rc;
  if (!X || !aligned(X, (uintptr_t)elem_bytes(dt))) return kErrInvalid;
  p->dt = dt;
  p->f8 = f8;
  p->rows = (uint32_t)rows;
  p->K = (uint32_t)K;
  p->KB = (uint32_t)((K + 127) / 128);
  p->KW = (uint32_t)((K + 511) / 512);
  p->sh = block_rows == 128 ? 7u : 0u;
  return kOk;
}

int plan_f8_gemm(const void* A, const void* As, int a_block_rows, const void* B, const void* Bs, int b_block_rows,
                 const void* bias, const void* R, const void* Z, const void* C, int64_t M, int64_t N, int64_t K,
                 uint32_t dtypes, int act, F8GemmPlan* p) {
  if (!p || M < 0 || N < 0 || K < 0) return kErrInvalid;
  if (act < 0 || act > 5) return kErrInvalid;
  if ((a_block_rows != 1 && a_block_rows != 128) || (b_block_rows != 1 && b_block_rows != 128)) return kErrInvalid;
  const int a = (int)(dtypes & 0xffu), b = (int)((dtypes >> 8) & 0xffu);
  const int dtb = (int)((dtypes >> 16) & 0xffu), out = (int)((dtypes >> 24) & 0xffu & ~(uint32_t)kSumsF32);
  p->wide = ((dtypes >> 24) & (uint32_t)kSumsF32) != 0;
  if (!valid_f8(a) || !valid_f8(b) || !valid_float_dt(out) || (bias && !valid_float_dt(dtb))) return kErrUnsupported;
  if (M >= kMaxBytes || N >= kMaxBytes || K >= kMaxBytes) return kErrUnsupported;
  const int64_t so = elem_bytes(out);
  p->empty = M == 0 || N == 0;
  if (p->empty) return kOk;
  if (too_large(N * so, M) || (bias && too_large(N, elem_bytes(dtb)))) return kErrUnsupported;
  int64_t ab, asb, bb, bsb;
  int rc = check_packed(A, As, M, K, a_block_rows, &ab, &asb);
  if (rc) return rc;
  rc = check_packed(B, Bs, N, K, b_block_rows, &bb, &bsb);
  if (rc) return rc;
  if (!C || !aligned(C, (uintptr_t)so) || (R && !aligned(R, (uintptr_t)so)) || (Z && !aligned(Z, (uintptr_t)so))) return kErrInvalid;
  if (Z && (Z == C || Z == R)) return kErrInvalid;     // R is read again after Z is written
  if (bias && !aligned(bias, (uintptr_t)elem_bytes(dtb))) return kErrInvalid;
  p->fa = a;
  p->fb = b;
  p->dto = out;
  p->bias_dt = bias ? dtb : -1;
  p->M = (uint32_t)M;
  p->N = (uint32_t)N;
  p->KB = (uint32_t)((K + 127) / 128);
  p->KW = (uint32_t)((K + 511) / 512);
  p->ash = a_block_rows == 128 ? 7u : 0u;
  p->bsh = b_block_rows == 128 ? 7u : 0u;
  p->a_bytes = (uint32_t)ab;
  p->as_bytes = (uint32_t)asb;
  p->b_bytes = (uint32_t)bb;
  p->bs_bytes = (uint32_t)bsb;
  p->bias_bytes = bias ? (uint32_t)(N * elem_bytes(dtb)) : 0u;
  p->c_bytes = (uint32_t)(M * N * so);
  return kOk;
}

}  // namespace biasact
