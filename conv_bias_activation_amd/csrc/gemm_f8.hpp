// gemm_f8.hpp — fused product of two 8-bit operands on gfx950, few rows:
//   C[M,N] = act(A[M,K] . B[N,K]^T + bias[N] (+ R[M,N]))
//
// Streaming kernel.  A wave holds a block of 16 NB rows of B (n) by 16 MB rows
// of A (m) and walks its part of k; the workgroup's waves split k and add their
// sums through LDS at the end, in wave order, so every result has one fixed
// order of additions.
//
// k advances by blocks of 128, one v_mfma_scale_f32_16x16x128 each: lane (r, g)
// takes the chunks of 16 codes g and 4 + g of row r (any assignment will do that
// is the same for both operands, since a block has one scale), straight from
// memory, so that a load covers 64 consecutive bytes of each of 16 rows and the
// next one the rest of the same cache lines.
#pragma once

#include "gemm_f8_tile.hpp"

namespace biasact {

// NB, MB: blocks of 16 rows of B and A per wave; NW: waves along k; UN: blocks of
// k that a wave has under way.
template <int FA, int FB, int DTO, int NB, int MB, int NW, int UN>
__global__ __launch_bounds__(64 * NW) void f8_stream_kernel(F8GemmArgs a) {
  constexpr int TN = 16 * NB, TM = 16 * MB;
  // the waves' sums, [m][n] with n contiguous and 4 floats of padding a row,
  // which keeps the rows of one access on different banks
  constexpr int LDR = TN + 4, SUMS = TM * LDR * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * SUMS];

  // neighbouring workgroups of an XCD share rows of B
  const uint32_t t = xcd_contiguous(blockIdx.x, gridDim.x);
  const uint32_t tn = t / a.tiles_m, tm = t - tn * a.tiles_m;
  const uint32_t n0 = tn * TN, m0 = tm * TM;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = lane & 15, g = lane >> 4;        // the matrix instructions' lane layout

  // Rows past the end are not stored: they read as zeros, or as whatever row a
  // huge offset wraps to.
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes), rbs = make_rsrc(a.Bs, a.bs_bytes);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes), ras = make_rsrc(a.As, a.as_bytes);

  // this wave's blocks of k: d0 .. d1 - 1
  const uint32_t per = (a.KB + NW - 1) / NW;
  const uint32_t d0 = min(w * per, a.KB), d1 = min(d0 + per, a.KB);

  f8::Frag bf[UN][NB], af[UN][MB];
  uint32_t bs[UN][NB], as[UN][MB];
  auto load = [&](int u, uint32_t d) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t row = n0 + 16 * i + r, at = (row * a.KB + d) * 128u + g * 16u;
      bf[u][i].lo = ld_b128(rb, at);
      bf[u][i].hi = ld_b128(rb, at + 64u);
      bs[u][i] = ld_b8(rbs, (row >> a.bsh) * a.KW * 4u + d);
    }
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const uint32_t row = m0 + 16 * j + r, at = (row * a.KB + d) * 128u + g * 16u;
      af[u][j].lo = ld_b128(ra, at);
      af[u][j].hi = ld_b128(ra, at + 64u);
      as[u][j] = ld_b8(ras, (row >> a.ash) * a.KW * 4u + d);
    }
  };
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (d0 + u < d1) load(u, d0 + u);

  // ---- bias and residual of this thread's outputs, under the main loop -----------------
  // quad o (four consecutive n of one row) of the tile, o = threadIdx.x + 64 NW p
  constexpr int QUADS = TM * TN / 4, P = (QUADS + 64 * NW - 1) / (64 * NW);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes), rz = make_rsrc(a.Z, a.Z ? a.c_bytes : 0u);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  const bool vec = a.N % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R) |
                                     reinterpret_cast<uintptr_t>(a.Z)) & (4u * Elem<DTO>::bytes - 1u)) == 0;
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
  f32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t d = d0; d < d1; d += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (d + u < d1) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < MB; ++j)
            if constexpr (DTO == DT_F32) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    f8::widen_part<FB>(bf[u][i], q, f8::scale_field(bs[u][i], 0)),
                    f8::widen_part<FA>(af[u][j], q, f8::scale_field(as[u][j], 0)), acc[i][j], 0, 0, 0);
            } else {
              acc[i][j] = f8::mfma16<FB, FA>(bf[u][i], af[u][j], acc[i][j], bs[u][i], as[u][j]);
            }
        __builtin_amdgcn_sched_barrier(0);           // (loads ahead of the products would need registers of their own)
        if (d + u + UN < d1) load(u, d + u + UN);
      }
  }

  // ---- sums of the waves, epilogue ---------------------------------------------------
  // accumulator register e of lane (r, g): n = 16 i + 4 g + e, m = 16 j + r
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
      for (int e = 0; e < 4; ++e) z[e] += add[p][e];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mx::act<ACT, DTO>(z[e], a.alpha);
      if (vec) {
        if (a.Z) store4<DTO>(rz, at[p], true, z[0], z[1], z[2], z[3]);
        store4<DTO>(rc, at[p], true, y[0], y[1], y[2], y[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (a.Z) store1<DTO>(rz, at[p] + e, n0 + nl + e < a.N, z[e]);
          store1<DTO>(rc, at[p] + e, n0 + nl + e < a.N, y[e]);
        }
      }
    }
  });
}

template <int DTO, int NB, int MB>
inline void launch_f8_stream(F8GemmArgs a, hipStream_t s) {
  constexpr int NW = 8;
  a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  a.tiles_m = (a.M + 16 * MB - 1) / (16 * MB);
  note_launch("gemm fp8 stream, %d n x %d m, k over %d waves", 16 * NB, 16 * MB, NW);
  f8::with_formats(a.fa, a.fb, [&](auto fa_c, auto fb_c) {
    launch_kernel(f8_stream_kernel<decltype(fa_c)::value, decltype(fb_c)::value, DTO, NB, MB, NW, (NB * MB > 4 ? 1 : 2)>,
                  dim3(a.tiles_m * a.tiles_n), dim3(64 * NW), s, a);
  });
}

inline uint64_t tiles_of(const F8GemmArgs& a, uint32_t bm, uint32_t bn) {
  return (uint64_t)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn);
}

// K = 0 (no blocks) runs the streaming kernel, whose waves then have nothing to add.
template <int DTO>
inline void launch_gemm_f8(const F8GemmArgs& a, hipStream_t s) {
  const uint64_t blocks = tiles_of(a, 64, 64);
  if (a.KB > 0 && blocks > 256) {
    const uint64_t t128 = tiles_of(a, 128, 128);
    const uint64_t small = t128 <= 256 ? 15 : (t128 + 511) / 512 * 24, large = (tiles_of(a, 256, 256) + 255) / 256 * 40;
    if constexpr (DTO != DT_F32)                       // (which has no registers for widened operands)
      if (large < small) return launch_f8_tile<DTO, 2, 4, 4, 2>(a, s);
    return launch_f8_tile<DTO, 2, 2, 2, 2>(a, s);
  }
  if (a.M <= 16) return launch_f8_stream<DTO, 1, 1>(a, s);
  if (a.M <= 32) return launch_f8_stream<DTO, 2, 2>(a, s);
  launch_f8_stream<DTO, 4, 4>(a, s);
}

}  // namespace biasact
