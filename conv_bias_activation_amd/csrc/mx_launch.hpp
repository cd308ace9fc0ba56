// mx_launch.hpp — launch entry points of the MXFP4 kernels (one translation
// unit per A type).  Return 0, or -1 for an unknown type.
#pragma once

#include <hip/hip_runtime.h>

#include "mx_args.hpp"

namespace biasact {

int launch_mx_quant(int dt, const MxQuantArgs& a, bool rows, bool back, hipStream_t s);
int launch_gemm_mx_mxfp4(int dto, const MxGemmArgs& a, hipStream_t s);
int launch_gemm_mx_f16(int dto, const MxGemmArgs& a, hipStream_t s);
int launch_gemm_mx_bf16(int dto, const MxGemmArgs& a, hipStream_t s);

}  // namespace biasact
