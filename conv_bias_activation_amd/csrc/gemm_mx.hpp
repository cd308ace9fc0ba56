// gemm_mx.hpp — fused product with an MXFP4 right operand on gfx950:
//   C[M,N] = act(A[M,K] . B[N,K]^T + bias[N] (+ R[M,N]))
// B in MXFP4 (mx_args.hpp), A in MXFP4, fp16 or bf16.
//
// Streaming kernel.  A wave holds a block of 16 NB rows of B (n) by 16 MB rows
// of A (m) and walks k; the workgroup's waves take turns along k and add their
// sums through LDS at the end, in wave order, so every result has one fixed
// order of additions.  Operands go from global memory straight to registers;
// a piece's registers are loaded anew, for a later group, as soon as its
// matrix instructions are issued.
//
// k advances by groups of 128.  Lane L (row r = L % 16, g = L / 16) loads 16
// bytes of codes, block g of its row's group, so one load covers 64
// consecutive bytes of each of 16 rows, and the group's four scale bytes as
// one word.
//   MXFP4 A: v_mfma_scale_f32_16x16x128 takes the blocks as they lie, each lane
//     with its own scale (byte g of the word, shifted down).
//   16-bit A: four 4x4 transpositions across the lanes of a row (two half-wave
//     and two row swaps) turn the block per lane into dword g of each of the
//     four blocks: matrix instruction c then covers the 32 k of block c, lane g
//     the eight from 8 g on, and A's loads too cover 64 consecutive bytes a row.
//     The codes become bf16 values with their scale (exact: two significant
//     bits and bf16's fp32 exponent range) for v_mfma_f32_16x16x32_bf16.
//   fp16 A: while every scale of a group lies in 2^-13 .. 2^13 its values are
//     normal fp16 numbers and go to v_mfma_f32_16x16x32_f16.  Otherwise A's
//     values are split into bf16 parts x = hi + lo, exactly (11 significant
//     bits into 8 + 3), with an instruction for each.
#pragma once

#include "epilogue.hpp"
#include "launch_kernel.hpp"
#include "mx_args.hpp"
#include "mx_launch.hpp"
#include "tile_map.hpp"

namespace biasact {

typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace mx {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// acc += (codes a) . (codes b)^T over 128 k, one block of 32 a lane, its scale
// in byte 0 of the scale words
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 acc, uint32_t sa, uint32_t sb) {
  const i32x8 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Register c of lane (r, g) becomes register g of lane (r, c).
__device__ __forceinline__ void transpose_groups(u32x4& v) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {        // upper half of a <-> lower half of b
    const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = s[0];
    b = s[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {        // odd 16-lane rows of a <-> even rows of b
    const auto s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = s[0];
    b = s[1];
  };
  uint32_t d0 = v.x, d1 = v.y, d2 = v.z, d3 = v.w;
  swap32(d0, d2);
  swap32(d1, d3);
  swap16(d0, d1);
  swap16(d2, d3);
  v = u32x4{d0, d1, d2, d3};
}

// eight codes -> bf16 with their scale (exponent field of s)
__device__ __forceinline__ u32x4 decode_bf16(uint32_t c, float s) {
  u32x4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  return v;
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                 acc, 0, 0, 0);
}

// eight codes -> fp16 with their scale
__device__ __forceinline__ u32x4 decode_f16(uint32_t c, float s) {
  u32x4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3));
  return v;
}

__device__ __forceinline__ f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0,
                                                0, 0);
}

// Two fp16 values as bf16 pairs: hi = x rounded to 8 significant bits, lo the
// rest.  An infinity keeps its hi part alone (the rest would be NaN).
__device__ __forceinline__ void split_f16(uint32_t w, uint32_t& hi, uint32_t& lo) {
  uint32_t h[2], l[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float x = widen<DT_F16>((w >> (16 * e)) & 0xffffu);
    h[e] = narrow<DT_BF16>(x);
    const float d = x - widen<DT_BF16>(h[e]);
    l[e] = __builtin_fabsf(x) == __builtin_inff() ? 0u : narrow<DT_BF16>(d);
  }
  hi = h[0] | (h[1] << 16);
  lo = l[0] | (l[1] << 16);
}

// Eight 16-bit values; p need only be aligned for one.
__device__ __forceinline__ u32x4 load_x8(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Eight values shifted down by d of them, zeros from above; d >= 8: all zero.
__device__ __forceinline__ u32x4 shift_x8(u32x4 v, uint32_t d) {
  const bool odd = d & 1u, two = d & 2u, four = d & 4u, all = d >= 8u;
  v = odd ? u32x4{__builtin_amdgcn_alignbit(v.y, v.x, 16), __builtin_amdgcn_alignbit(v.z, v.y, 16),
                  __builtin_amdgcn_alignbit(v.w, v.z, 16), v.w >> 16} : v;
  v = two ? u32x4{v.y, v.z, v.w, 0u} : v;
  v = four ? u32x4{v.z, v.w, 0u, 0u} : v;
  return all ? u32x4{0u, 0u, 0u, 0u} : v;
}

// The activation for an output of type DTO (fp32 GELU keeps its subnormal tail).
template <int ACT, int DTO>
__device__ __forceinline__ float act(float z, float alpha) {
  if constexpr (ACT == ACT_GELU && DTO == DT_F32) return gelu_f32_tail(z);
  else return act_fn<ACT, DTO>(z, alpha);
}

}  // namespace mx

// NB, MB: blocks of 16 rows of B and A per wave; NW: waves along k; UN: groups
// of 128 k that a wave has under way.
template <int DTA, int DTO, int NB, int MB, int NW, int UN>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(MxGemmArgs a) {
  constexpr int TN = 16 * NB, TM = 16 * MB;
  // partial sums of one wave, [m][n] with n contiguous; 4 floats of padding a
  // row keep the rows that one store instruction covers on different banks
  constexpr int LDR = TN + 4;
  __shared__ __attribute__((aligned(16))) float red[NW][TM][LDR];

  // neighbouring workgroups of an XCD share rows of B
  const uint32_t t = xcd_contiguous(blockIdx.x, gridDim.x);
  const uint32_t tn = t / a.tiles_m, tm = t - tn * a.tiles_m;
  const uint32_t n0 = tn * TN, m0 = tm * TM;
  const int lane = threadIdx.x & 63;
  const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, g = lane >> 4;

  // Rows past the end are not stored: those of packed operands read as zeros or
  // as whatever row their offset wraps to, those of a 16-bit A repeat its last.
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes), rbs = make_rsrc(a.Bs, a.bs_bytes);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes), ras = make_rsrc(a.As, a.as_bytes);
  const uint8_t* A = static_cast<const uint8_t*>(a.A);
  const uint32_t wrow = (n0 + r) * a.G, mrow = (m0 + r) * a.G;
  uint32_t xrow[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) xrow[j] = min(m0 + 16 * j + r, a.M - 1) * a.K;

  // UN groups under way: codes and scales of B, 16-byte pieces (and scales) of A
  constexpr int XC = DTA == DT_MXFP4 ? 1 : 4;
  u32x4 wc[UN][NB], xc[UN][MB][XC];
  uint32_t ws[UN][NB], xs[UN][MB];
  auto load_w = [&](int u, uint32_t q) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t at = wrow + (16u * i * a.G + q);
      wc[u][i] = ld_b128(rb, at * 64u + 16u * g);
      ws[u][i] = ld_b32(rbs, at * 4u);
    }
  };
  // Piece c of A: values 128 q + 32 c + 8 g .. + 7 of each row; where that runs
  // past K (>= 8 for a 16-bit A), the row's last eight, shifted down on use.
  auto load_x = [&](int u, int c, uint32_t q) {
    if constexpr (DTA == DT_MXFP4) {
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const uint32_t at = mrow + (16u * j * a.G + q);
        xc[u][j][0] = ld_b128(ra, at * 64u + 16u * g);
        xs[u][j] = ld_b32(ras, at * 4u);
      }
    } else {
      const uint32_t k = min(q * 128u + c * 32u + g * 8u, a.K - 8u);
#pragma unroll
      for (int j = 0; j < MB; ++j) xc[u][j][c] = mx::load_x8(A + (size_t)((xrow[j] + k) * 2u));
    }
  };

  f32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Adds group q's products from slot u and loads group q + UN NW into it.
  auto multiply = [&](int u, uint32_t q) {
    const uint32_t qn = q + UN * NW;
    const bool more = qn < a.G;                        // uniform
    if constexpr (DTA == DT_MXFP4) {
      uint32_t sx[MB];
#pragma unroll
      for (int j = 0; j < MB; ++j) sx[j] = xs[u][j] >> (8 * g);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = mx::mfma_mx(wc[u][i], xc[u][j][0], acc[i][j], ws[u][i] >> (8 * g), sx[j]);
      if (more) {
        load_w(u, qn);
        load_x(u, 0, qn);
      }
    } else {
      u32x4 wv[NB];
      uint32_t sw[NB];
      bool normal = DTA == DT_F16;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        wv[i] = wc[u][i];
        sw[i] = ws[u][i];
      }
      // (the widest fp16 block has no registers for the next codes beside these:
      // it loads them last)
      constexpr bool LATE = DTA == DT_F16 && NB * MB == 16;
      if (more && !LATE) load_w(u, qn);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        mx::transpose_groups(wv[i]);
        if constexpr (DTA == DT_F16)                   // 2^-13 .. 2^13: 0.5 and 6 times it are normal in fp16
#pragma unroll
          for (int c = 0; c < 4; ++c) normal = normal && ((sw[i] >> (8 * c)) & 255u) - 114u <= 26u;
      }
      if constexpr (DTA == DT_F16) normal = __all(normal);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if ((q + 1) * 128u > a.K) {                    // uniform: the row ends in this group
          const uint32_t k = q * 128u + c * 32u + g * 8u;
#pragma unroll
          for (int j = 0; j < MB; ++j) xc[u][j][c] = mx::shift_x8(xc[u][j][c], k - min(k, a.K - 8u));
        }
        auto scale = [&](int i) { return __uint_as_float(((sw[i] >> (8 * c)) & 255u) << 23); };
        if constexpr (DTA == DT_BF16) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const u32x4 v = mx::decode_bf16(wv[i][c], scale(i));
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = mx::mfma_bf16(v, xc[u][j][c], acc[i][j]);
          }
        } else if (normal) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const u32x4 v = mx::decode_f16(wv[i][c], scale(i));
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = mx::mfma_f16(v, xc[u][j][c], acc[i][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < MB; ++j) {
            __builtin_amdgcn_sched_barrier(0);         // one row block's parts at a time: there are no more registers
            u32x4 hi, lo;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              uint32_t h, l;
              mx::split_f16(xc[u][j][c][d], h, l);
              hi[d] = h;
              lo[d] = l;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              uint32_t codes = wv[i][c];
              asm volatile("" : "+v"(codes));          // decoded anew for each j, not kept: registers again
              const u32x4 v = mx::decode_bf16(codes, scale(i));
              acc[i][j] = mx::mfma_bf16(v, hi, acc[i][j]);
              acc[i][j] = mx::mfma_bf16(v, lo, acc[i][j]);
            }
          }
        }
        if (more) load_x(u, c, qn);
      }
      if (more && LATE) load_w(u, qn);
    }
  };

  // ---- the first groups of this wave -----------------------------------------------
  const uint32_t q0 = UN * w;
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (q0 + u < a.G) {
      load_w(u, q0 + u);
#pragma unroll
      for (int c = 0; c < XC; ++c) load_x(u, c, q0 + u);
    }

  // ---- bias and residual of this thread's outputs, under the main loop ----------
  // quad o (four consecutive n of one row) of the tile, o = threadIdx.x + 64 NW p
  constexpr int QUADS = TM * TN / 4, P = (QUADS + 64 * NW - 1) / (64 * NW);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  const bool vec = a.N % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R)) &
                                    (4u * Elem<DTO>::bytes - 1u)) == 0;
  float add[P][4];
  uint32_t at[P];                                      // element offset of the quad, or kOOB
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t o = threadIdx.x + 64 * NW * p, ml = o / (TN / 4), nl = (o - ml * (TN / 4)) * 4;
    const uint32_t m = m0 + ml, n = n0 + nl;
    const bool in = o < (uint32_t)QUADS && m < a.M && n < a.N;
    at[p] = in ? m * a.N + n : kOOB;
    uint32_t idx[4] = {n, n + 1, n + 2, n + 3};
    load_bias_vec<4>(a.bias, a.bias_bytes, a.bias_dt, idx, in ? a.N : 0u, add[p]);
    if (a.R) {
      float rv[4];
      if (vec) {
        load4<DTO>(rr, at[p], in, rv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) rv[e] = load1<DTO>(rr, at[p] + e, in && n + e < a.N);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) add[p][e] += rv[e];
    }
  }

  // ---- main loop -------------------------------------------------------------------
  for (uint32_t q = q0; q < a.G; q += UN * NW) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (q + u < a.G) multiply(u, q + u);
  }

  // ---- sums of the waves, epilogue ---------------------------------------------------
  // accumulator register e of lane (r, g): n = 16 i + 4 g + e, m = 16 j + r
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) *reinterpret_cast<f32x4*>(&red[w][16 * j + r][16 * i + 4 * g]) = acc[i][j];
  __syncthreads();
  with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act_c)::value;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (at[p] == kOOB) continue;
      const uint32_t o = threadIdx.x + 64 * NW * p, ml = o / (TN / 4), nl = (o - ml * (TN / 4)) * 4;
      f32x4 z = *reinterpret_cast<const f32x4*>(&red[0][ml][nl]);
#pragma unroll
      for (int v = 1; v < NW; ++v) z += *reinterpret_cast<const f32x4*>(&red[v][ml][nl]);
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mx::act<ACT, DTO>(z[e] + add[p][e], a.alpha);
      if (vec) {
        store4<DTO>(rc, at[p], true, y[0], y[1], y[2], y[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store1<DTO>(rc, at[p] + e, n0 + nl + e < a.N, y[e]);
      }
    }
  });
}

// A 16-bit A of fewer than eight columns (no 16-byte piece of a row to load),
// or no columns at all: one lane per output, its few products in turn.
template <int DTA, int DTO>
__global__ __launch_bounds__(256) void mx_short_kernel(MxGemmArgs a) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  if (at >= a.M * a.N) return;
  const uint32_t m = at / a.N, n = at - m * a.N;
  float z = 0.0f;
  if constexpr (DTA != DT_MXFP4) {
    for (uint32_t k = 0; k < a.K; ++k) {
      const float x = widen<DTA>(static_cast<const uint16_t*>(a.A)[m * a.K + k]);
      const uint32_t c = static_cast<const uint8_t*>(a.B)[n * 64u + (k >> 1)] >> (4 * (k & 1));
      const float s = __uint_as_float((uint32_t) static_cast<const uint8_t*>(a.Bs)[n * 4u] << 23);
      z += x * __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0)[0];
    }
  }
  if (a.bias_dt >= 0) z += load_bias(make_rsrc(a.bias, a.bias_bytes), a.bias_dt, n);
  if (a.R) z += load1<DTO>(make_rsrc(a.R, a.c_bytes), at, true);
  with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
    store1<DTO>(make_rsrc(a.C, a.c_bytes), at, true, mx::act<decltype(act_c)::value, DTO>(z, a.alpha));
  });
}

template <int DTA, int DTO>
inline void launch_mx_short(const MxGemmArgs& a, hipStream_t s) {
  note_launch("gemm mxfp4, k < 8");
  launch_kernel(mx_short_kernel<DTA, DTO>, dim3((a.M * a.N + 255) / 256), dim3(256), s, a);
}

template <int DTA, int DTO, int NB, int MB, int NW>
inline void launch_mx_stream(MxGemmArgs a, hipStream_t s) {
  // as many groups under way as leave room for the sums and the current one
  constexpr int GROUP = 5 * NB + (DTA == DT_MXFP4 ? 5 : 16) * MB, LEFT = 150 - 4 * NB * MB;
  constexpr int UN = 4 * GROUP <= LEFT ? 4 : 2 * GROUP <= LEFT ? 2 : 1;
  a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  a.tiles_m = (a.M + 16 * MB - 1) / (16 * MB);
  note_launch("gemm mxfp4 stream, %d n x %d m, k over %d waves", 16 * NB, 16 * MB, NW);
  launch_kernel(mx_stream_kernel<DTA, DTO, NB, MB, NW, UN>, dim3(a.tiles_m * a.tiles_n), dim3(64 * NW), s, a);
}

}  // namespace biasact
