// gemm_mx.hpp — fused product with an MXFP4 right operand on gfx950:
//   C[M,N] = act(A[M,K] . B[N,K]^T + bias[N] (+ R[M,N]))
// B in MXFP4 (mx_args.hpp), A in MXFP4, fp16 or bf16.
//
// Streaming kernel.  A wave holds a block of 16 NB rows of B (n) by 16 MB rows
// of A (m) and walks its part of k; the workgroup's waves split k and add their
// sums through LDS at the end, in wave order, so every result has one fixed
// order of additions.
//
// k advances by units of two groups of 128.  Eight neighbouring lanes load 128
// consecutive bytes, a cache line, of one row: a load then touches 8 lines,
// where the layout of the matrix instructions (lanes r, r + 16, r + 32, r + 48
// share row r) would touch 64, and a CU reads from L2 at 133 GB/s instead of 68
// with half lines and 30 with quarters of them.  Each wave turns that into the
// instruction's layout through LDS of its own, a row's 16-byte chunk c at slot
// c ^ (row & 7) so that neither side meets a bank twice; a wave's LDS operations
// run in order, so this needs no barrier.  A register is loaded anew, for the
// next unit or piece, as soon as it has gone to LDS.  Scale words come for
// two units at a time, one row a lane.
//   MXFP4 A: v_mfma_scale_f32_16x16x128, lane (r, g) with block g of row r and
//     its scale (byte g of the word, shifted down).
//   16-bit A: v_mfma_f32_16x16x32 c covers block c, lane (r, g) the eight k from
//     8 g on.  For bf16 the codes become bf16 values with their scale, which is
//     exact (two significant bits and bf16's fp32 exponent range; the smallest,
//     2^-128, is a subnormal, which the instruction takes) up to scale byte 252,
//     where 6 times the scale is 1.5 * 2^127.  Past that (bytes 253 and 254, which
//     the quantiser never writes) a value can be infinite, and then so is, or NaN,
//     every sum of its row: a wave that ends with such sums and has such scales
//     forms its sums anew, each block's products unscaled and then scaled in fp32.
//     (The loop itself has no registers for a second way, and looking for the
//     bytes in it took 1 to 2 % of the small products' time.)  For fp16
//     they become fp16 values with their scale while every scale in sight lies
//     in 2^-13 .. 2^13 (0.5 and 6 times it are normal fp16 numbers); else each
//     block's products are summed unscaled and scaled in fp32.  In sight are the
//     scales of the wave's rows in a group; byte 0, of a block of zeros or read for
//     rows past N, takes the second way too: 1x4096x4096 5.8 us, 6.6 with one zero
//     block in a thousand, 1x4095x4096 7.3 (64 rows: 9.9, 11.0 and 12.0).
//
// Measured with N = K = 4096, bf16 outputs: two MXFP4 operands 4.4 us for 8 rows
// of A and 5.6 for 64; a bf16 A 5.3 us for one row (9 MB, 1.9 us at 4.9 TB/s),
// 9.8 for 64 and 15.5 for 256 (554 TFLOP/s).  With few rows that is a launch
// (1.7 us for a trivial kernel), fetching the code, and the loads' latency; with
// many, a CU's reads of A and B from L2 (640 KB for 256 rows, 4.8 us) and their
// way through LDS (4.5 us), which the two waves of a SIMD overlap only in part.
// Tiles of 64x64 that share no operand between waves need the fewest LDS bytes
// per product; sixteen waves along k changed these times by 1 %.
#pragma once

#include "epilogue.hpp"
#include "launch_kernel.hpp"
#include "mx_act.hpp"
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

// 2^(b - 127), NaN for 255, as fp32
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// Orders a wave's LDS accesses before and after (the hardware runs them in
// order; this keeps the compiler from exchanging them).
__device__ __forceinline__ void lds_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Eight values shifted down by d of them, zeros from above; d >= 8: all zero.
__device__ __forceinline__ u32x4 shift_x8(u32x4 v, uint32_t d) {
  const bool odd = d & 1u, two = d & 2u, four = d & 4u, all = d >= 8u;
  v = odd ? u32x4{__builtin_amdgcn_alignbit(v.y, v.x, 16), __builtin_amdgcn_alignbit(v.z, v.y, 16),
                  __builtin_amdgcn_alignbit(v.w, v.z, 16), v.w >> 16} : v;
  v = two ? u32x4{v.y, v.z, v.w, 0u} : v;
  v = four ? u32x4{v.z, v.w, 0u, 0u} : v;
  return all ? u32x4{0u, 0u, 0u, 0u} : v;
}

}  // namespace mx

// NB, MB: blocks of 16 rows of B and A per wave; NW: waves along k; UN: units of
// 256 k that a wave has under way.
template <int DTA, int DTO, int NB, int MB, int NW, int UN>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(MxGemmArgs a) {
  constexpr int TN = 16 * NB, TM = 16 * MB;
  constexpr bool LATE = NB * MB == 16;                 // the widest block: every register counts
  // Per wave: one unit of B, one piece (MXFP4: unit) of A, 2 KB per 16 rows, and
  // two units' scale words; at the end the waves' sums, [m][n] with n contiguous
  // and 4 floats of padding a row, which keeps the rows of one access on
  // different banks.
  constexpr int LDR = TN + 4;
  constexpr int SROWS = TN + (DTA == DT_MXFP4 ? TM : 0);
  constexpr int W_AT = 0, X_AT = NB * 2048, S_AT = X_AT + MB * 2048, WAVE = S_AT + SROWS * 16;
  constexpr int SUMS = TM * LDR * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * (WAVE > SUMS ? WAVE : SUMS)];

  // neighbouring workgroups of an XCD share rows of B
  const uint32_t t = xcd_contiguous(blockIdx.x, gridDim.x);
  const uint32_t tn = t / a.tiles_m, tm = t - tn * a.tiles_m;
  const uint32_t n0 = tn * TN, m0 = tm * TM;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, g = lane >> 4;        // the matrix instructions' lane layout
  const uint32_t lr = lane >> 3, lc = lane & 7;       // the loads': row (and row + 8), 16-byte chunk
  uint8_t* const my = smem + w * WAVE;
  const uint32_t put = lr * 128u + ((lc ^ lr) << 4);  // a loaded chunk's place; row + 8: 1024 further
  const uint32_t get = r * 128u, sw = r & 7;          // row r's chunk c: get + ((c ^ sw) << 4)

  // Rows past the end are not stored: they read as zeros, or as whatever row a
  // huge offset wraps to.
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes), rbs = make_rsrc(a.Bs, a.bs_bytes);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes), ras = make_rsrc(a.As, a.as_bytes);
  const uint32_t wrow = (n0 + lr) * a.G, mrow = (m0 + lr) * (DTA == DT_MXFP4 ? a.G : a.K);

  // this wave's units of k: d0 .. d1 - 1
  const uint32_t units = (a.G + 1) >> 1, per = (units + NW - 1) / NW;
  const uint32_t d0 = min(w * per, units), d1 = min(d0 + per, units);

  // under way: UN units of codes of B (and of A), XS pieces of 64 k of a 16-bit A
  constexpr int XS = 2 * UN, XC = DTA == DT_MXFP4 ? UN : XS;
  u32x4 wc[UN][NB][2], xc[XC][MB][2];
  // unit d of a packed operand; with an odd G the last one's second group is zero
  auto load_packed = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, uint32_t d, auto& v) __attribute__((always_inline)) {
    const bool cut = 2 * d + 1 >= a.G && lc >= 4;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v) / sizeof(v[0])); ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[i][h] = ld_b128(rs, cut ? kOOB : (row + ((16u * i + 8u * h) * a.G + 2 * d)) * 64u + 16u * lc);
  };
  // Piece p of a 16-bit A: values 64 p + 8 lc .. + 7 of each row; where that runs
  // past K (>= 8), the row's last eight, shifted down on use.  (A row need only be
  // aligned for one value: the GPU runs with unaligned access on.)
  auto load_x = [&](int slot, uint32_t p) __attribute__((always_inline)) {
    const uint32_t k = min(p * 64u + lc * 8u, a.K - 8u);
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) xc[slot][j][h] = ld_b128(ra, (mrow + ((16u * j + 8u * h) * a.K + k)) * 2u);
  };
  // Scale words of groups q .. q + 3 (zero past the row's end): row n0 + lane of B
  // for the first 16 NB lanes, and row m0 + lane of an MXFP4 A.
  auto load_s = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, uint32_t q) {
    u32x4 v = {0, 0, 0, 0};
    const uint32_t at = (row * a.G + q) * 4u;
    if (q + 4 <= a.G) {                                // uniform
      v = ld_b128(rs, at);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 3; ++e)
        if (q + e < a.G) v[e] = ld_b32(rs, at + e * 4u);
    }
    return v;
  };
  u32x4 sb = {0, 0, 0, 0}, sa = {0, 0, 0, 0};
  auto load_scales = [&](uint32_t q) {
    sb = load_s(rbs, n0 + min(lane, TN - 1u), q);
    if constexpr (DTA == DT_MXFP4) sa = load_s(ras, m0 + min(lane, TM - 1u), q);
  };
  auto put_scales = [&] {
    if (lane < TN) *reinterpret_cast<u32x4*>(my + S_AT + lane * 16u) = sb;
    if constexpr (DTA == DT_MXFP4)
      if (lane < TM) *reinterpret_cast<u32x4*>(my + S_AT + (TN + lane) * 16u) = sa;
  };

  f32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Adds unit d's products from slot u and loads unit d + UN into it.
  auto multiply = [&](int u, uint32_t d) __attribute__((always_inline)) {
    const bool more = d + UN < d1;                     // uniform
    const uint32_t word0 = ((d - d0) & 1u) * 2u;       // of the scale words at hand
    mx::lds_order();
    if (word0 == 0) {
      put_scales();
      if (d + 2 < d1) load_scales(2 * d + 4);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4*>(my + W_AT + i * 2048 + h * 1024 + put) = wc[u][i][h];
    if (more) load_packed(rb, wrow, d + UN, wc[u]);
    if constexpr (DTA == DT_MXFP4) {
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4*>(my + X_AT + j * 2048 + h * 1024 + put) = xc[u][j][h];
      if (more) load_packed(ra, mrow, d + UN, xc[u]);
      mx::lds_order();
#pragma unroll
      for (int half = 0; half < 2; ++half) {           // (a missing second group adds zeros)
        u32x4 xf[MB];
        uint32_t sx[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          xf[j] = *reinterpret_cast<const u32x4*>(my + X_AT + j * 2048 + get + (((4 * half + g) ^ sw) << 4));
          sx[j] = *reinterpret_cast<const uint32_t*>(my + S_AT + (TN + 16 * j + r) * 16 + (word0 + half) * 4) >> (8 * g);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const u32x4 wf =
              *reinterpret_cast<const u32x4*>(my + W_AT + i * 2048 + get + (((4 * half + g) ^ sw) << 4));
          const uint32_t ws =
              *reinterpret_cast<const uint32_t*>(my + S_AT + (16 * i + r) * 16 + (word0 + half) * 4) >> (8 * g);
#pragma unroll
          for (int j = 0; j < MB; ++j) acc[i][j] = mx::mfma_mx(wf, xf[j], acc[i][j], ws, sx[j]);
        }
      }
    } else {
#pragma unroll UN
      for (int half = 0; half < 2; ++half) {
        const uint32_t q = 2 * d + half;
        if (half == 1 && q >= a.G) continue;           // uniform
        mx::lds_order();
        uint32_t ws[NB];                               // the four blocks' scale bytes of row 16 i + r
        bool normal = true;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          ws[i] = *reinterpret_cast<const uint32_t*>(my + S_AT + (16 * i + r) * 16 + (word0 + half) * 4);
          if constexpr (DTA == DT_F16)
#pragma unroll
            for (int c = 0; c < 4; ++c)                // (padding past K holds zeros, whatever its scale)
              normal = normal && (((ws[i] >> (8 * c)) & 255u) - 114u <= 26u || q * 128u + c * 32u >= a.K);
        }
        if constexpr (DTA == DT_F16) normal = __all(normal);
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
          const int slot = UN == 1 ? pp : 2 * half + pp;
          const uint32_t p = 2 * q + pp;
          if ((q + 1) * 128u > a.K) {                  // uniform: the row ends in this group
            const uint32_t k = p * 64u + lc * 8u, over = k - min(k, a.K - 8u);
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) xc[slot][j][h] = mx::shift_x8(xc[slot][j][h], over);
          }
          mx::lds_order();
#pragma unroll
          for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<u32x4*>(my + X_AT + j * 2048 + h * 1024 + put) = xc[slot][j][h];
          if (p + XS < 4 * d1) load_x(slot, p + XS);
          mx::lds_order();
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int c = 2 * pp + cc;                 // block of the group
            u32x4 xf[MB];
            uint32_t wf[NB];                           // codes of the eight k from 8 g on
#pragma unroll
            for (int i = 0; i < NB; ++i)
              wf[i] = *reinterpret_cast<const uint32_t*>(my + W_AT + i * 2048 + get + (((4 * half + c) ^ sw) << 4) + 4 * g);
#pragma unroll
            for (int j = 0; j < MB; ++j)
              xf[j] = *reinterpret_cast<const u32x4*>(my + X_AT + j * 2048 + get + (((4 * cc + g) ^ sw) << 4));
            auto field = [&](int i) { return __uint_as_float(((ws[i] >> (8 * c)) & 255u) << 23); };
            if constexpr (DTA == DT_BF16) {
#pragma unroll
              for (int i = 0; i < NB; ++i) {
                const u32x4 v = mx::decode_bf16(wf[i], field(i));
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mx::mfma_bf16(v, xf[j], acc[i][j]);
              }
            } else if (normal) {
#pragma unroll
              for (int i = 0; i < NB; ++i) {
                const u32x4 v = mx::decode_f16(wf[i], field(i));
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mx::mfma_f16(v, xf[j], acc[i][j]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < NB; ++i) {
                const u32x4 v = mx::decode_f16(wf[i], 1.0f);
                float s[4];                            // of the sums' rows, 16 i + 4 g + e
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  s[e] = mx::scale_value(my[S_AT + (16 * i + 4 * g + e) * 16 + (word0 + half) * 4 + c]);
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                  const f32x4 z = mx::mfma_f16(v, xf[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[e], s[e], acc[i][j][e]);
                }
              }
            }
          }
        }
      }
    }
  };

  // ---- the first units of this wave --------------------------------------------------
  if (d0 < d1) load_scales(2 * d0);
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (d0 + u < d1) {
      load_packed(rb, wrow, d0 + u, wc[u]);
      if constexpr (DTA == DT_MXFP4) load_packed(ra, mrow, d0 + u, xc[u]);
    }
  if constexpr (DTA != DT_MXFP4) {
#pragma unroll
    for (int p = 0; p < XS; ++p)
      if (d0 < d1) load_x(p, 4 * d0 + p);              // (a unit has four pieces)
  }

  // ---- bias and residual of this thread's outputs -----------------------------------
  // under the main loop, or after it where that has no registers for them
  // quad o (four consecutive n of one row) of the tile, o = threadIdx.x + 64 NW p
  constexpr int QUADS = TM * TN / 4, P = (QUADS + 64 * NW - 1) / (64 * NW);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  const bool vec = a.N % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R)) &
                                    (4u * Elem<DTO>::bytes - 1u)) == 0;
  float add[P][4];
  uint32_t at[P];                                      // element offset of the quad, or kOOB
  auto load_add = [&] {
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
  };
  if constexpr (!LATE) load_add();

  // ---- main loop -------------------------------------------------------------------
  for (uint32_t d = d0; d < d1; d += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (d + u < d1) multiply(u, d + u);
  }

  // ---- once more, block by block, where a scale was more than bf16 can take ----------
  if constexpr (DTA == DT_BF16) {
    float t = 0.0f;                                    // NaN with any sum that is not finite
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) t = __builtin_fmaf(acc[i][0][e], 0.0f, t);
    uint32_t high = 0;                                 // bit 7 of a byte: a scale byte was 253 or 254
    if (__builtin_expect(__any(t != 0.0f), 0)) {
#pragma unroll 1
      for (uint32_t q = 2 * d0; q < min(2 * d1, a.G); ++q)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint32_t s = ld_b32(rbs, ((n0 + 16 * i + r) * a.G + q) * 4u);
          // from 253 on a byte's lower bits reach 125 and bit 7 is set; 255 (NaN) has both low bits
          high |= ((s & 0x7f7f7f7fu) + 0x03030303u) & s & ~((s << 7) & (s << 6));
        }
    }
    if (__builtin_expect(__any((high & 0x80808080u) != 0), 0)) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (uint32_t b = 8 * d0; b < min(8 * d1, 4 * a.G); ++b) {     // blocks of the row
        const uint32_t k = b * 32u + g * 8u, from = min(k, a.K - 8u);
        u32x4 xf[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) xf[j] = mx::shift_x8(ld_b128(ra, ((m0 + 16 * j + r) * a.K + from) * 2u), k - from);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const u32x4 v = mx::decode_bf16(ld_b32(rb, (n0 + 16 * i + r) * a.G * 64u + b * 16u + g * 4u), 1.0f);
          float s[4];                                  // of the sums' rows, 16 i + 4 g + e
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = mx::scale_value(ld_b8(rbs, (n0 + 16 * i + 4 * g + e) * a.G * 4u + b));
#pragma unroll
          for (int j = 0; j < MB; ++j) {
            const f32x4 z = mx::mfma_bf16(v, xf[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(z[e], s[e], acc[i][j][e]);
          }
        }
      }
    }
  }

  if constexpr (LATE) load_add();

  // ---- sums of the waves, epilogue ---------------------------------------------------
  // accumulator register e of lane (r, g): n = 16 i + 4 g + e, m = 16 j + r
  __syncthreads();                                     // the sums go over every wave's operands
  auto sum = [&](uint32_t v, uint32_t ml, uint32_t nl) {
    return reinterpret_cast<f32x4*>(smem + v * SUMS + (ml * LDR + nl) * 4u);
  };
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) *sum(w, 16 * j + r, 16 * i + 4 * g) = acc[i][j];
  __syncthreads();
  with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act_c)::value;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (at[p] == kOOB) continue;
      const uint32_t o = threadIdx.x + 64 * NW * p, ml = o / (TN / 4), nl = (o - ml * (TN / 4)) * 4;
      f32x4 z = *sum(0, ml, nl);
#pragma unroll
      for (int v = 1; v < NW; ++v) z += *sum(v, ml, nl);
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
    // fp32 holds 6 times the scale up to byte 252: the last factor of 2 or 4 of
    // bytes 253 and 254 comes after the product with x
    const uint32_t byte = a.K ? static_cast<const uint8_t*>(a.Bs)[n * 4u] : 0u;     // (nothing there for no columns)
    const bool high = byte == 253u || byte == 254u;
    const float s = __uint_as_float((high ? 252u : byte) << 23), rest = byte == 253u ? 2.0f : 4.0f;
    for (uint32_t k = 0; k < a.K; ++k) {
      const float x = widen<DTA>(static_cast<const uint16_t*>(a.A)[m * a.K + k]);
      const uint32_t c = static_cast<const uint8_t*>(a.B)[n * 64u + (k >> 1)] >> (4 * (k & 1));
      const float v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0)[0];
      z = high ? __builtin_fmaf(x * v, rest, z) : __builtin_fmaf(x, v, z);
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

template <int DTA, int DTO, int NB, int MB>
inline void launch_mx_stream(MxGemmArgs a, hipStream_t s) {
  constexpr int NW = 8;
  a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  a.tiles_m = (a.M + 16 * MB - 1) / (16 * MB);
  note_launch("gemm mxfp4 stream, %d n x %d m, k over %d waves", 16 * NB, 16 * MB, NW);
  const dim3 grid(a.tiles_m * a.tiles_n), block(64 * NW);
  // Two units under way where a wave walks at least four, for which B comes in at
  // the rate that its loads under way allow: one row by 4096x16384 (bf16) 13.4 us,
  // with one unit 16.8.  A shorter product takes longer with two, which unroll the
  // code that it has to fetch: 17x4096x4096 7.6 us with two, 6.6 with one.
  if constexpr (NB * MB <= 2)
    if (a.G >= 2 * NW * 4)
      return launch_kernel(mx_stream_kernel<DTA, DTO, NB, MB, NW, 2>, grid, block, s, a);
  launch_kernel(mx_stream_kernel<DTA, DTO, NB, MB, NW, 1>, grid, block, s, a);
}

}  // namespace biasact
