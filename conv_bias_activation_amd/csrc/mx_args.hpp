// mx_args.hpp — kernel argument blocks of the MXFP4 operators.
//
// MXFP4: a value is a 4-bit code (sign, 2-bit exponent, 1-bit mantissa: 0,
// 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times the scale of its block,
// 32 consecutive values along the reduction index k.  The scale is one byte b
// for 2^(b - 127); b = 255 is NaN.  A row of K values is stored as whole
// groups of 128: 64 bytes of codes (even k in the low four bits) and 4 scale
// bytes per group, the padding zero.
#pragma once

#include <stdint.h>

#include "device_common.hpp"

namespace biasact {

enum : int { DT_MXFP4 = 5 };

// C[M,N] = act(A . B^T + bias (+ R)), B in MXFP4, A in MXFP4 or 16-bit.
struct MxGemmArgs {
  const void* A;           // [M, K] 16-bit, or codes [M, 64 G]
  const void* As;          // scales [M, 4 G] of an MXFP4 A, else null
  const void* B;           // codes [N, 64 G]
  const void* Bs;          // scales [N, 4 G]
  const void* bias;
  const void* R;           // residual [M, N] in C's type, or null
  void* C;
  uint32_t M, N, K, G;     // G = ceil(K / 128)
  uint32_t a_bytes, as_bytes, b_bytes, bs_bytes, bias_bytes, c_bytes;
  int bias_dt;             // DT_* of bias, or -1 without bias
  int act;
  float alpha;
  uint32_t tiles_m, tiles_n;
};

struct MxQuantArgs {
  const void* X;           // [rows, K] (k_axis 1) or [K, rows] (k_axis 0); the output of dequantisation
  void* codes;             // [rows, 64 G]
  void* scales;            // [rows, 4 G]
  uint32_t rows, K, G;
  uint32_t total;          // k_axis 1: 8-value chunks, rows * 16 G
  FastDiv div_row;         // by 16 G
  FastDiv div_tiles;       // k_axis 0: by the column tiles, ceil(rows / 64)
};

}  // namespace biasact
