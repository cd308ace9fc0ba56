// norm_args.hpp — kernel argument blocks and launch entry points of layer norm
// and of the gradients of layer norm and of the bias-and-activation epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace biasact {

struct NormArgs {
  const void* X;           // [rows, N]
  const void* gamma;       // [N], or null (ones)
  const void* beta;        // [N], or null (zeros)
  void* Y;                 // [rows, N]
  float* mean;             // [rows], or null
  float* rstd;             // [rows], or null
  uint32_t rows, N;
  int dtw;                 // DT_* of gamma and beta
  float eps;
};

struct NormGradArgs {
  const void* dY;          // [rows, N]
  const void* X;           // [rows, N]
  const void* gamma;       // [N], or null (ones)
  const float* mean;       // [rows]
  const float* rstd;       // [rows]
  void* dX;                // [rows, N]
  float* part;             // [parts][2][N] column sums of dY * xhat and of dY, or null
  uint32_t rows, N, parts;
  int dtw;                 // DT_* of gamma
};

struct ActGradArgs {
  const void* dY;          // [M, N]
  const void* Z;           // [M, N]; null with act none
  void* dZ;                // [M, N], or null
  float* part;             // [parts][N] column sums of dZ, or null
  uint32_t M, N, parts;
  uint32_t lane_bits;      // log2 of the lanes that share a row
  int act;
  float alpha;
};

// Sums over the parts of P[parts][stride] columns 0 .. n - 1 -> out in dt.
struct JoinArgs {
  const float* part;
  void* out[2];            // columns 0 .. n - 1 and n .. 2 n - 1; either may be null
  uint32_t parts, n, stride;
  int dt;
};

int launch_layer_norm_f32(int dty, const NormArgs& a, hipStream_t s);
int launch_layer_norm_f16(int dty, const NormArgs& a, hipStream_t s);
int launch_layer_norm_bf16(int dty, const NormArgs& a, hipStream_t s);
int launch_layer_norm_grad_f32(int dty, const NormGradArgs& a, hipStream_t s);
int launch_layer_norm_grad_f16(int dty, const NormGradArgs& a, hipStream_t s);
int launch_layer_norm_grad_bf16(int dty, const NormGradArgs& a, hipStream_t s);
int launch_act_grad(int dt, const ActGradArgs& a, hipStream_t s);
void launch_join_columns(const JoinArgs& a, hipStream_t s);

}  // namespace biasact
