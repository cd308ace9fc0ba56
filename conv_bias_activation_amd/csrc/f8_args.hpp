// f8_args.hpp — kernel argument blocks of the 8-bit floating-point operators.
//
// A value is an 8-bit code (OCP e4m3: 4 exponent and 3 mantissa bits, largest
// 448, no infinity; or e5m2: 5 and 2, largest 57344) times the scale of its
// block: 128 consecutive values along the reduction index k, of one row or of
// 128 rows.  The scale is one byte b for 2^(b - 127); b = 255 is NaN.  A row of
// K values is stored as whole blocks: 128 * KB bytes of codes, KB = ceil(K / 128),
// the padding zero, and a row of scales as whole words: 4 * KW bytes, KW = ceil(K / 512).
#pragma once

#include <stdint.h>

#include "device_common.hpp"

namespace biasact {

enum : int { DT_E4M3 = 6, DT_E5M2 = 7 };

// C[M,N] = act(A . B^T + bias (+ R)), both operands in 8 bits.
struct F8GemmArgs {
  const void* A;           // codes [M, 128 KB]
  const void* As;          // scales [M >> ash, 4 KW] (rounded up)
  const void* B;           // codes [N, 128 KB]
  const void* Bs;          // scales [N >> bsh, 4 KW] (rounded up)
  const void* bias;
  const void* R;           // residual [M, N] in C's type, or null
  void* Z;                 // the sums before the activation, in C's type, or null
  void* C;
  uint32_t M, N, KB, KW;
  uint32_t ash, bsh;       // 0: a scale for each row, 7: for 128 rows
  uint32_t a_bytes, as_bytes, b_bytes, bs_bytes, bias_bytes, c_bytes;
  int fa, fb;              // DT_E4M3 or DT_E5M2
  int bias_dt;             // DT_* of bias, or -1 without bias
  int act;
  float alpha;
  uint32_t tiles_m, tiles_n;
};

struct F8QuantArgs {
  const void* X;           // [rows, K] (k_axis 1) or [K, rows] (k_axis 0); the output of dequantisation
  void* codes;             // [rows, 128 KB]
  void* scales;            // [rows >> sh, 4 KW] (rounded up)
  uint32_t rows, K, KB, KW;
  uint32_t sh;             // 0: a scale for each row, 7: for 128 rows
  FastDiv div;             // the kernel's inner count of work items
};

}  // namespace biasact
