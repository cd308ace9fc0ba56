// norm_plan.hpp — how the rows of the gradient kernels are divided, which the
// workspaces' sizes follow (host and kernels' launches; no device code).
#pragma once

#include <stdint.h>

namespace biasact {

// Rows longer than this are read again for each step of a layer norm; up to it
// a row stays in its threads' registers.
constexpr uint32_t kNormLong = 16384u;

// Threads that share a row of N values in layer_norm_grad (16 to 1024), and the
// rows that a workgroup of 256 or more then takes at once: eight or sixteen values a
// thread, whose column sums, weights and next row just fit its registers.
inline uint32_t norm_grad_threads(uint32_t N) {
  return N <= 128u ? 16u : N <= 1024u ? 64u : N <= 4096u ? 256u : N <= 8192u ? 512u : 1024u;
}
inline uint32_t norm_grad_rows_at_once(uint32_t N) {
  const uint32_t t = norm_grad_threads(N);
  return t >= 256u ? 1u : 256u / t;
}

// Workgroups that each keep the column sums of their share of the rows: two a CU, or
// one, whose next row is under way while it works on this one, where a row of X and dY
// takes 32 KB (pair_bytes: of a value of each) or more than 4096 values (us with 256
// and 512: 32768x4096 bf16 153 to 170 and 156, fp32 285 and 304, 4096x16384 bf16 96 and 110,
// 8192x5120 48 and 54; 32768x1024 42 and 37, 32768x256 27 and 20, 8192x1280 fp32 32
// and 28; with 1024 more but for 32768x256, 22).
inline uint32_t norm_grad_parts(uint32_t rows, uint32_t N, uint32_t pair_bytes) {
  if (N > kNormLong) return rows < 64u ? rows : 64u;
  const uint32_t once = norm_grad_rows_at_once(N), groups = (rows + once - 1) / once;
  const uint32_t most = N <= 4096u && N * pair_bytes < 32768u ? 512u : 256u;
  return groups < most ? groups : most;
}

// Lanes (as a power of two) that share a row of N values in bias_act_grad, eight
// columns a lane, and the row splits for M rows: up to 1024 workgroups, four a CU (us,
// bf16: 8192x16384 GELU 163, with 512 200, 2048 167, 4096 167; 32768x4096 LeakyReLU 151, with
// 2048 165, 4096 168).
inline uint32_t act_grad_lane_bits(uint32_t N) {
  uint32_t b = 0;
  while (b < 6u && (8u << b) < N) ++b;
  return b;
}
inline uint32_t act_grad_parts(uint32_t M, uint32_t N) {
  const uint32_t b = act_grad_lane_bits(N), tiles = (N + (8u << b) - 1) / (8u << b);
  const uint32_t once = 256u >> b;                     // rows that a workgroup takes at once
  const uint32_t groups = (M + once - 1) / once, want = (1024u + tiles - 1) / tiles;
  return groups < want ? groups : want;
}

}  // namespace biasact
