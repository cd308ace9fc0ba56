// api_f8.hip — the extern "C" entry points of the 8-bit floating-point operators
// (include/biasact.h).  Each call checks its arguments (plan_f8.cpp), then queues
// one kernel on the caller's stream.  Nothing is allocated or synchronised here.
#include "biasact.h"
#include "f8_launch.hpp"
#include "launch_kernel.hpp"
#include "plan.hpp"

using namespace biasact;

namespace {

int quant_impl(const void* X, const void* codes, const void* scales, int64_t rows, int64_t K, int k_axis,
               int block_rows, uint32_t dtypes, bool back, hipStream_t s) {
  F8QuantPlan p;
  const int rc = plan_f8_quant(X, codes, scales, rows, K, k_axis, block_rows, dtypes, &p);
  if (rc || p.empty) return rc;
  F8QuantArgs a;
  a.X = X;
  a.codes = const_cast<void*>(codes);
  a.scales = const_cast<void*>(scales);
  a.rows = p.rows;
  a.K = p.K;
  a.KB = p.KB;
  a.KW = p.KW;
  a.sh = p.sh;
  a.div = make_fastdiv(1);         // set with the kernel
  if (launch_f8_quant(p.dt, p.f8, a, k_axis == 1, back, s)) return kErrUnsupported;
  return launch_status();
}

int gemm_impl(const void* A, const void* As, int a_block_rows, const void* B, const void* Bs, int b_block_rows,
              const void* bias, const void* R, void* Z, void* C, int64_t M, int64_t N, int64_t K, uint32_t dtypes,
              int act, float alpha, hipStream_t s) {
  F8GemmPlan p;
  const int rc = plan_f8_gemm(A, As, a_block_rows, B, Bs, b_block_rows, bias, R, Z, C, M, N, K, dtypes, act, &p);
  if (rc || p.empty) return rc;
  F8GemmArgs a;
  a.A = A;
  a.As = As;
  a.B = B;
  a.Bs = Bs;
  a.bias = bias;
  a.R = R;
  a.Z = Z;
  a.C = C;
  a.M = p.M;
  a.N = p.N;
  a.KB = p.KB;
  a.KW = p.KW;
  a.ash = p.ash;
  a.bsh = p.bsh;
  a.a_bytes = p.a_bytes;
  a.as_bytes = p.as_bytes;
  a.b_bytes = p.b_bytes;
  a.bs_bytes = p.bs_bytes;
  a.bias_bytes = p.bias_bytes;
  a.c_bytes = p.c_bytes;
  a.fa = p.fa;
  a.fb = p.fb;
  a.bias_dt = p.bias_dt;
  a.act = act;
  a.alpha = alpha;
  a.tiles_m = a.tiles_n = 0;       // set with the tile
  switch (p.dto) {
    case DT_F32: launch_gemm_f8_f32(a, s); break;
    case DT_F16: p.wide ? launch_gemm_f8_wide_f16(a, s) : launch_gemm_f8_f16(a, s); break;
    default: p.wide ? launch_gemm_f8_wide_bf16(a, s) : launch_gemm_f8_bf16(a, s); break;
  }
  return launch_status();
}

}  // namespace

extern "C" {

int fp8_packed_size(int64_t rows, int64_t K, int block_rows, size_t* codes_bytes, size_t* scales_bytes) {
  int64_t c, s;
  if (!codes_bytes || !scales_bytes) return kErrInvalid;
  const int rc = f8_sizes(rows, K, block_rows, &c, &s);
  if (rc) return rc;
  *codes_bytes = (size_t)c;
  *scales_bytes = (size_t)s;
  return kOk;
}

int fp8_quantize(const void* X, void* codes, void* scales, int64_t rows, int64_t K, int k_axis, int block_rows,
                 uint32_t dtypes, hipStream_t stream) {
  return quant_impl(X, codes, scales, rows, K, k_axis, block_rows, dtypes, false, stream);
}

int fp8_dequantize(const void* codes, const void* scales, void* Y, int64_t rows, int64_t K, int k_axis, int block_rows,
                   uint32_t dtypes, hipStream_t stream) {
  return quant_impl(Y, codes, scales, rows, K, k_axis, block_rows, dtypes, true, stream);
}

int gemm_fp8_bias_act(const void* A, const void* a_scales, int a_block_rows, const void* B, const void* b_scales,
                      int b_block_rows, const void* bias, void* Z, void* C, int64_t M, int64_t N, int64_t K,
                      uint32_t dtypes, int act, float alpha, hipStream_t stream) {
  return gemm_impl(A, a_scales, a_block_rows, B, b_scales, b_block_rows, bias, nullptr, Z, C, M, N, K, dtypes, act, alpha, stream);
}

int gemm_fp8_bias_add_act(const void* A, const void* a_scales, int a_block_rows, const void* B, const void* b_scales,
                          int b_block_rows, const void* bias, const void* R, void* Z, void* C, int64_t M, int64_t N,
                          int64_t K, uint32_t dtypes, int act, float alpha, hipStream_t stream) {
  if (!R && M > 0 && N > 0) return kErrInvalid;
  return gemm_impl(A, a_scales, a_block_rows, B, b_scales, b_block_rows, bias, R, Z, C, M, N, K, dtypes, act, alpha, stream);
}

}  // extern "C"
