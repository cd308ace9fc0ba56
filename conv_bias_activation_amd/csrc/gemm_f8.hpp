// gemm_f8.hpp — fused product of two 8-bit operands on gfx950, few rows:
//   C[M,N] = act(A[M,K] . B[N,K]^T + bias[N] (+ R[M,N]))
//
// Streaming kernel.  A wave holds a block of 16 NB rows of B (n) by 16 MB rows
// of A (m) and walks its part of k; the workgroup's waves split k and add their
// sums through LDS at the end, in wave order, so every result has one fixed
// order of additions.
//
// k advances by blocks of 128, one v_mfma_scale_f32_16x16x128 each.  Codes go to LDS
// of the wave's own without passing through registers, eight lanes a row of 128
// bytes, UN blocks under way (a register of each would allow two); chunk c of row
// r lies at slot c ^ (r / 2 % 8).  Lane (r, g) takes the chunks g and 4 + g of row r:
// any assignment will do that is the same for both operands, since a block has one scale.
//
// Bound by the latency of loads and by reading B: 8x4096x4096 bf16 takes 4.2 us with B in the
// last-level cache and 6.1 with B out of it, whose 16.8 MB are 3.4 us at a large copy's
// 4.9 TB/s; 16x4096x4096 4.7 and 6.5; with Z, a residual and GELU 4.5 and 4.9.  (From
// that cache: 16x4096x16384 12.7, 8x16384x4096 12.4.)  With 3 or 4 blocks under way the LDS
// holds one workgroup a CU: 8x4096x4096 4.3, 32x4096x4096 7.7 instead of 6.6; blocks dealt
// to the waves in turn made no difference.  With fp32 sums 8x4096x4096 4.3,
// 32x4096x4096 5.6 (5.3).
#pragma once

#include "gemm_f8_tile.hpp"

namespace biasact {

// NB, MB: blocks of 16 rows of B and A per wave; NW: waves along k; UN: blocks of
// k that a wave has under way.  WIDE: sums in fp32 throughout (gemm_f8_tile.hpp).
template <int FA, int FB, int DTO, bool WIDE, int NB, int MB, int NW, int UN>
__global__ __launch_bounds__(64 * NW) void f8_stream_kernel(F8GemmArgs a) {
  constexpr int TN = 16 * NB, TM = 16 * MB;
  // the waves' sums, [m][n] with n contiguous and 4 floats of padding a row,
  // which keeps the rows of one access on different banks
  constexpr int SUMS = TM * (TN + 4) * 4, STAGE = (TN + TM) * 128;
  static_assert(NW * UN * STAGE <= 160 * 1024 && SUMS <= UN * STAGE, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * UN * STAGE];

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

  // block d into stage u: lane l fills slot l % 8 of row l / 8 of each eight rows; the
  // swizzle of the odd eights differs by 4, i.e. by 64 bytes of the row
  uint8_t* const my = smem + w * (UN * STAGE);
  const uint32_t chunk = ((lane & 7u) ^ ((lane >> 4) & 3u)) * 16u;
  const uint32_t b_off = (n0 + (lane >> 3)) * a.KB * 128u + chunk, a_off = (m0 + (lane >> 3)) * a.KB * 128u + chunk;
  uint32_t bs[UN][NB], as[UN][MB];
  auto load = [&](int u, uint32_t d) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(my + u * STAGE + i * 1024), 16,
                                               (b_off ^ (64u * (i & 1))) + (8u * i * a.KB + d) * 128u, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 2 * MB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(my + u * STAGE + (2 * NB + j) * 1024), 16,
                                               (a_off ^ (64u * (j & 1))) + (8u * j * a.KB + d) * 128u, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i) bs[u][i] = ld_b8(rbs, ((n0 + 16 * i + r) >> a.bsh) * a.KW * 4u + d);
#pragma unroll
    for (int j = 0; j < MB; ++j) as[u][j] = ld_b8(ras, ((m0 + 16 * j + r) >> a.ash) * a.KW * 4u + d);
  };
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (d0 + u < d1) load(u, d0 + u);

  SumEpilogue<DTO, TM, TN, NW, 64 * NW> out;
  out.load(a, m0, n0);                                 // under the main loop

  // ---- main loop -------------------------------------------------------------------
  f32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t get = r * 128u + ((g ^ ((r >> 1) & 7u)) << 4);   // chunk 4 + g: 64 bytes away
  for (uint32_t d = d0; d < d1; d += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (d + u < d1) {
        // this block's loads have landed: those of later blocks may be under way
        __builtin_amdgcn_sched_barrier(0);
        if (d + u + UN - 1 < d1) __builtin_amdgcn_s_waitcnt(f8::wait_vm((UN - 1) * 3 * (NB + MB)));
        else __builtin_amdgcn_s_waitcnt(f8::wait_vm(0));
        __builtin_amdgcn_sched_barrier(0);
        auto frag = [&](int at) __attribute__((always_inline)) {
          const uint8_t* p = my + u * STAGE + at * 2048;
          return f8::Frag{*reinterpret_cast<const u32x4*>(p + get), *reinterpret_cast<const u32x4*>(p + (get ^ 64u))};
        };
        f8::Frag af[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) af[j] = frag(NB + j);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const f8::Frag bf = frag(i);
#pragma unroll
          for (int j = 0; j < MB; ++j)
            if constexpr (WIDE) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8::widen_part<FB>(bf, q, f8::scale_field(bs[u][i], 0)),
                                                                    f8::widen_part<FA>(af[j], q, f8::scale_field(as[u][j], 0)),
                                                                    acc[i][j], 0, 0, 0);
            } else {
              acc[i][j] = f8::mfma16<FB, FA>(bf, af[j], acc[i][j], bs[u][i], as[u][j]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);             // (the stage is read)
        if (d + u + UN < d1) load(u, d + u + UN);
      }
  }

  // ---- sums of the waves, epilogue ---------------------------------------------------
  // accumulator register e of lane (r, g): n = 16 i + 4 g + e, m = 16 j + r
  __syncthreads();                                     // the sums go over every wave's operands
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
      *reinterpret_cast<f32x4*>(smem + w * SUMS + ((16 * j + r) * (TN + 4) + 16 * i + 4 * g) * 4u) = acc[i][j];
  __syncthreads();
  out.store(a, smem, n0);
}

template <int DTO, bool WIDE, int NB, int MB, int UN>
inline void launch_f8_stream(F8GemmArgs a, hipStream_t s) {
  constexpr int NW = 8;
  a.tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
  a.tiles_m = (a.M + 16 * MB - 1) / (16 * MB);
  note_launch("gemm fp8 stream, %d n x %d m, k over %d waves%s", 16 * NB, 16 * MB, NW, WIDE ? ", fp32 sums" : "");
  f8::with_formats(a.fa, a.fb, [&](auto fa_c, auto fb_c) {
    launch_kernel(f8_stream_kernel<decltype(fa_c)::value, decltype(fb_c)::value, DTO, WIDE, NB, MB, NW, UN>,
                  dim3(a.tiles_m * a.tiles_n), dim3(64 * NW), s, a);
  });
}

// Choice of the kernel: the least estimated time.  Each kernel's workgroups take
// the 256 CUs in rounds, and a round takes a part of its own and one for each
// block of k.  The estimates, in 10 ns, fit these measurements (us, bf16 outputs,
// operands from the last-level cache):
//   stream 16x16          8x4096x4096 4.2, 16x4096x16384 12.7, 64x4096x4096 10.9, 256x4096x1024 15.9
//   stream 32 n x 16 m    32x4096x4096 5.3, 64x4096x4096 9.0
//   wave   64 m x 32 n    64x4096x4096 7.1, 256x4096x4096 13.6, 64x1024x16384 16.4
//   wave   64x64          64x4096x4096 9.1, 256x4096x4096 10.6, 256x4096x8192 17.3, 512x4096x4096 20.1
//   tile   64x64          64x4096x512 4.5, 256x4096x1024 5.5, 256x4096x4096 10.1, 256x4096x8192 18.2,
//                         1001x1503x333 5.9 (128x128: 6.9), 512x4096x4096 15.4, 1024x4096x1024 11.7
//   tile   128x128 deep   256x4096x4096 15.7, 512x4096x4096 16.4, 1024x4096x4096 21.0
//   tile   128x128 twice  1024x4096x1024 8.3, 1024x4096x4096 24.4, 2048x4096x4096 35, 4096x4096x128 13.5
//   tile   256x256        1024x4096x4096 38, 2048x4096x4096 41, 4096x4096x4096 57, 4096x4096x128 11.3
// (wave: each wave of four has a part of k; tile 64x64: two waves, four stages, two
// workgroups a CU; deep: one workgroup a CU with four stages, for products of one
// round, whose step would else be a load's latency: 4096x1024x32768 124, two stages
// 180; twice: two workgroups a CU.)
inline uint64_t f8_tiles(const F8GemmArgs& a, uint32_t bm, uint32_t bn) {
  return (uint64_t)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn);
}

enum { kF8Stream16, kF8Stream32, kF8Wave32, kF8Wave64, kF8Tile64, kF8TileDeep, kF8TileTwice, kF8TileLarge };

inline int f8_choice(const F8GemmArgs& a, bool large) {
  const uint64_t k = a.KB;
  if (k == 0) return kF8TileTwice;                     // nothing to add; its grid takes any M and N
  const auto rounds = [](uint64_t tiles, uint64_t per) { return (tiles + per - 1) / per; };
  const uint64_t t16 = f8_tiles(a, 16, 16), t32 = f8_tiles(a, 16, 32), w32 = f8_tiles(a, 64, 32), w64 = f8_tiles(a, 64, 64);
  const uint64_t t128 = f8_tiles(a, 128, 128), t256 = f8_tiles(a, 256, 256);
  const uint64_t rest64 = w64 % 512, rest128 = t128 % 512, rest256 = t256 % 256;
  uint64_t cost[8];
  cost[kF8Stream16] = 250 + 7 * k + (t16 > 256 ? (t16 - 256) * (k > 11 ? 7 * k : 80) / 256 : 0);
  cost[kF8Stream32] = rounds(t32, 256) * (250 + 9 * k);
  cost[kF8Wave32] = rounds(w32, 256) * (370 + 10 * k);
  cost[kF8Wave64] = rounds(w64, 256) * (550 + 16 * k);
  cost[kF8Tile64] = w64 / 512 * (450 + 34 * k) + (rest64 == 0 ? 0 : rest64 <= 256 ? 390 + 19 * k : 450 + 34 * k);
  cost[kF8TileDeep] = rounds(t128, 256) * (500 + (t128 <= 128 ? 34 : 50) * k);
  cost[kF8TileTwice] = t128 / 512 * (500 + 95 * k) + (rest128 == 0 ? 0 : rest128 <= 256 ? 400 + 62 * k : 500 + 95 * k);
  cost[kF8TileLarge] = t256 / 256 * (1000 + 146 * k) + (rest256 == 0 ? 0 : rest256 <= 128 ? 900 + 92 * k : 1000 + 146 * k);
  int best = 0;
  for (int i = 1; i < (large ? 8 : 7); ++i)
    if (cost[i] < cost[best]) best = i;
  return best;
}

// (Widened operands leave no registers for the largest tile.)
template <int DTO, bool WIDE>
inline void launch_gemm_f8(const F8GemmArgs& a, hipStream_t s) {
  switch (f8_choice(a, !WIDE)) {
    case kF8Stream16: return launch_f8_stream<DTO, WIDE, 1, 1, 2>(a, s);
    case kF8Stream32: return launch_f8_stream<DTO, WIDE, 2, 1, 2>(a, s);
    case kF8Wave32: return launch_f8_tile<DTO, WIDE, 1, 1, 2, 1, 4, 2>(a, s);
    case kF8Wave64: return launch_f8_tile<DTO, WIDE, 1, 1, 2, 2, 4, 2>(a, s);
    case kF8Tile64: return launch_f8_tile<DTO, WIDE, 1, 2, 2, 1, 1, 4>(a, s);
    case kF8TileDeep:
      // A wave ahead for operands of 64 MB and more, of which a part at least has left the
      // last-level cache by the time they are used, and three columns of tiles or more
      // (with fewer, its shares leave out most of A's rows).  us, bf16, with operands that take turns
      // out of that cache, without and with it, and then the same in the cache:
      //   4096x1024x32768 157 and 147, 125 and 136; 1024x4096x16384 78 and 75, 66 and 71;
      //   2048x2048x16384 75 and 73, 65 and 69; 8192x512x16384 83 and 79, 66 and 71
      //   4 rows of tiles: 512x8192x16384 82 and 85, 67 and 72; 2: 256x16384x8192 52 and 53, 37 and 39
      //   2 columns: 16384x256x8192 53 and 53, 38 and 41; 1: 32768x128x8192 74 and 71, 50 and 60
      // In a backward pass, whose operands were just quantised, it gives 20 us (32768x4096x1024
      // with dW of 4096x1024x32768: 593 and 573).
      if (a.N > 256 && (uint64_t)a.a_bytes + a.b_bytes >= 1u << 26) return launch_f8_tile<DTO, WIDE, 2, 2, 2, 2, 1, 4, true>(a, s);
      return launch_f8_tile<DTO, WIDE, 2, 2, 2, 2, 1, 4>(a, s);
    case kF8TileTwice: return launch_f8_tile<DTO, WIDE, 2, 2, 2, 2, 1, 2>(a, s);
    default:
      if constexpr (!WIDE) launch_f8_tile<DTO, WIDE, 2, 4, 4, 2, 1, 2>(a, s);
  }
}

}  // namespace biasact
