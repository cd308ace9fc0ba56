// f8_launch.hpp — launch entry points of the 8-bit floating-point kernels (the
// products: one translation unit per output type and kind of sum).  Return 0, or -1 for an
// unknown type.
#pragma once

#include <hip/hip_runtime.h>

#include "f8_args.hpp"

namespace biasact {

int launch_f8_quant(int dt, int f8, const F8QuantArgs& a, bool along_rows, bool back, hipStream_t s);
void launch_gemm_f8_f32(const F8GemmArgs& a, hipStream_t s);      // (sums in fp32)
void launch_gemm_f8_f16(const F8GemmArgs& a, hipStream_t s);
void launch_gemm_f8_bf16(const F8GemmArgs& a, hipStream_t s);
void launch_gemm_f8_wide_f16(const F8GemmArgs& a, hipStream_t s);  // sums in fp32
void launch_gemm_f8_wide_bf16(const F8GemmArgs& a, hipStream_t s);

}  // namespace biasact
