// gemm_mx.hpp — fused product with an MXFP4 right operand on gfx950:
//   C[M,N] = act(A[M,K] . B[N,K]^T + bias[N] (+ R[M,N]))
// B in MXFP4 (mx_args.hpp), A in MXFP4, fp16 or bf16.
//
// Streaming kernel.  A wave holds a block of 16 NB rows of B (n) by 16 MB rows
// of A (m) and walks k; the workgroup's waves take turns along k and add their
// sums through LDS at the end, in wave order, so every result has one fixed
// order of additions.  Operands go from global memory straight to registers.
//
// One step is 512 values of k.  Lane L (row r = L % 16, g = L / 16) loads the
// 64 bytes of codes of group 4 s + g of its row, and that group's four scale
// bytes as one word: block i of all four groups feeds the i-th matrix
// instruction, which needs 32 consecutive k per lane and any four blocks as
// long as both operands bring the same ones.
//   MXFP4 A: v_mfma_scale_f32_16x16x128, both scales applied by the
//     instruction (its operand selector takes byte i of the scale words).
//   16-bit A: the lane's 32 codes become 32 bf16 values with their scale (all
//     exact: two significant bits and bf16's fp32 exponent range), for four
//     v_mfma_f32_16x16x32_bf16.  fp16 values of A are split into bf16 parts
//     x = hi + lo, also exactly (11 significant bits into 8 + 3), each with
//     its own instruction.
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

// acc += (codes a) . (codes b)^T over 4 blocks of 32, scale byte I of each word
template <int I>
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 acc, uint32_t sa, uint32_t sb) {
  const i32x8 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, I, (int)sa, I, (int)sb);
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

// The values k0 .. k0 + 7 of a 16-bit row of K (zero from K on); whole: known
// to be all there.  The row need only be aligned for one value.
__device__ __forceinline__ u32x4 load_x8(const uint8_t* row, uint32_t k0, uint32_t K, bool whole) {
  u32x4 v = {0, 0, 0, 0};
  if (whole || k0 + 8u <= K) {
    __builtin_memcpy(&v, row + (size_t)k0 * 2u, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e < K)
        v[e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + (size_t)(k0 + e) * 2u) << (16 * (e & 1));
  }
  return v;
}

// The activation for an output of type DTO (fp32 GELU keeps its subnormal tail).
template <int ACT, int DTO>
__device__ __forceinline__ float act(float z, float alpha) {
  if constexpr (ACT == ACT_GELU && DTO == DT_F32) return gelu_f32_tail(z);
  else return act_fn<ACT, DTO>(z, alpha);
}

}  // namespace mx

template <int DTA, int DTO, int NB, int MB, int NW>
__global__ __launch_bounds__(64 * NW) void mx_stream_kernel(MxGemmArgs a) {
  constexpr int TN = 16 * NB, TM = 16 * MB;
  // partial sums of one wave, [m][n] with n contiguous; 4 floats of padding a
  // row keep the 16 rows that one store instruction covers on different banks
  constexpr int LDR = TN + 4;
  __shared__ __attribute__((aligned(16))) float red[NW][TM][LDR];

  const uint32_t t = xcd_contiguous(blockIdx.x, gridDim.x);
  const uint32_t tn = t / a.tiles_m, tm = t - tn * a.tiles_m;
  const uint32_t n0 = tn * TN, m0 = tm * TM;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, g = lane >> 4;

  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes), rbs = make_rsrc(a.Bs, a.bs_bytes);
  uint32_t nrow[NB], mrow[MB];            // rows past the end repeat the last one; their sums are not stored
#pragma unroll
  for (int i = 0; i < NB; ++i) nrow[i] = min(n0 + 16 * i + r, a.N - 1);
#pragma unroll
  for (int i = 0; i < MB; ++i) mrow[i] = min(m0 + 16 * i + r, a.M - 1);

  f32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t steps = (a.G + 3) >> 2;
  for (uint32_t s = w; s < steps; s += NW) {
    const uint32_t q = 4 * s + g;                     // this lane's group of 128
    const bool ok = q < a.G;
    u32x4 wc[NB][4];
    uint32_t ws[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      ws[i] = ld_b32(rbs, ok ? (nrow[i] * a.G + q) * 4u : kOOB);
#pragma unroll
      for (int b = 0; b < 4; ++b) wc[i][b] = ld_b128(rb, ok ? (nrow[i] * a.G + q) * 64u + 16u * b : kOOB);
    }
    if constexpr (DTA == DT_MXFP4) {
      const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes), ras = make_rsrc(a.As, a.as_bytes);
      u32x4 xc[MB][4];
      uint32_t xs[MB];
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        xs[j] = ld_b32(ras, ok ? (mrow[j] * a.G + q) * 4u : kOOB);
#pragma unroll
        for (int b = 0; b < 4; ++b) xc[j][b] = ld_b128(ra, ok ? (mrow[j] * a.G + q) * 64u + 16u * b : kOOB);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          acc[i][j] = mx::mfma_mx<0>(wc[i][0], xc[j][0], acc[i][j], ws[i], xs[j]);
          acc[i][j] = mx::mfma_mx<1>(wc[i][1], xc[j][1], acc[i][j], ws[i], xs[j]);
          acc[i][j] = mx::mfma_mx<2>(wc[i][2], xc[j][2], acc[i][j], ws[i], xs[j]);
          acc[i][j] = mx::mfma_mx<3>(wc[i][3], xc[j][3], acc[i][j], ws[i], xs[j]);
        }
    } else {
      const bool whole = (s + 1) * 512u <= a.K;       // uniform: every value of this step is there
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        u32x4 xv[MB][4];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const uint8_t* row = static_cast<const uint8_t*>(a.A) + (size_t)mrow[j] * a.K * 2u;
#pragma unroll
          for (int c = 0; c < 4; ++c) xv[j][c] = mx::load_x8(row, q * 128u + b * 32u + c * 8u, a.K, whole);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const float sc = __uint_as_float(((ws[i] >> (8 * b)) & 255u) << 23);
          u32x4 wv[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) wv[c] = mx::decode_bf16(wc[i][b][c], sc);
#pragma unroll
          for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if constexpr (DTA == DT_BF16) {
                acc[i][j] = mx::mfma_bf16(wv[c], xv[j][c], acc[i][j]);
              } else {
                u32x4 hi, lo;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t h, l;
                  mx::split_f16(xv[j][c][e], h, l);
                  hi[e] = h;
                  lo[e] = l;
                }
                acc[i][j] = mx::mfma_bf16(wv[c], hi, acc[i][j]);
                acc[i][j] = mx::mfma_bf16(wv[c], lo, acc[i][j]);
              }
            }
        }
      }
    }
  }

  // accumulator register e of lane (r, g): n = 16 i + 4 g + e, m = 16 j + r
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) *reinterpret_cast<f32x4*>(&red[w][16 * j + r][16 * i + 4 * g]) = acc[i][j];
  __syncthreads();

  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  const __amdgpu_buffer_rsrc_t rbias = make_rsrc(a.bias, a.bias_bytes);
  with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act_c)::value;
    for (int o = threadIdx.x; o < TM * TN; o += 64 * NW) {
      const int ml = o / TN, nl = o - ml * TN;
      const uint32_t m = m0 + ml, n = n0 + nl;
      if (m >= a.M || n >= a.N) continue;
      float z = red[0][ml][nl];
#pragma unroll
      for (int v = 1; v < NW; ++v) z += red[v][ml][nl];
      if (a.bias_dt >= 0) z += load_bias(rbias, a.bias_dt, n);
      if (a.R) z += load1<DTO>(rr, m * a.N + n, true);
      store1<DTO>(rc, m * a.N + n, true, mx::act<ACT, DTO>(z, a.alpha));
    }
  });
}

template <int DTA, int DTO, int NB, int MB, int NW>
inline void launch_mx_stream(MxGemmArgs a, hipStream_t s) {
  a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  a.tiles_m = (a.M + 16 * MB - 1) / (16 * MB);
  note_launch("gemm mxfp4 stream, %d n x %d m, k over %d waves", 16 * NB, 16 * MB, NW);
  launch_kernel(mx_stream_kernel<DTA, DTO, NB, MB, NW>, dim3(a.tiles_m * a.tiles_n), dim3(64 * NW), s, a);
}

template <int DTA, int DTO>
inline void launch_gemm_mx_to(const MxGemmArgs& a, hipStream_t s) {
  if (a.M <= 16) launch_mx_stream<DTA, DTO, 1, 1, 4>(a, s);
  else launch_mx_stream<DTA, DTO, 4, 4, 4>(a, s);
}

template <int DTA>
inline int launch_gemm_mx(int dto, const MxGemmArgs& a, hipStream_t s) {
  switch (dto) {
    case DT_F32: launch_gemm_mx_to<DTA, DT_F32>(a, s); return 0;
    case DT_F16: launch_gemm_mx_to<DTA, DT_F16>(a, s); return 0;
    case DT_BF16: launch_gemm_mx_to<DTA, DT_BF16>(a, s); return 0;
    default: return -1;
  }
}

}  // namespace biasact
