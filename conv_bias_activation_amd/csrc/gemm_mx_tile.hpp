// gemm_mx_tile.hpp — tiled fused product of two MXFP4 operands on gfx950:
//   C[M,N] = act(A . B^T + bias (+ R)), both operands as rows of k (mx_args.hpp)
//
// Workgroup: 4 waves, 2 (m) x 2 (n), of SJ x SI accumulator blocks of 32x32
// each: an output tile of 64 SJ (m) x 64 SI (n).  A k-tile is one group of 128
// values, 64 bytes of codes and 4 scale bytes a row.  Two workgroups share a
// CU: one's loads, LDS reads, start and end run under the other's matrix
// instructions, v_mfma_scale_f32_32x32x64.
//
// Codes reach LDS without passing through registers, 16 bytes a lane, three
// stages deep; chunk c of row r lies at slot c ^ ((r >> 2) & 3), so the eight
// lanes that a 16-byte LDS read serves at a time are on different banks.  Half
// h of a wave takes chunks 2 h and 2 h + 1 of its rows: its two scale bytes
// are then neighbours, and one shift puts them where the instruction's operand
// selector reads byte 0 for the first k-step and byte 1 for the second.
// Scales travel 16 bytes a row for four k-tiles at once, through registers:
// fetched with each k-tile they would touch one cache line per row and tile,
// as many as the codes do.
//
// Epilogue: the fp32 sums leave through LDS, 32 SJ rows at a time (16-byte
// chunk c of row r at slot c ^ 2 (r & 15)), so every lane handles eight
// consecutive outputs of a row: one bias fetch for all its rows, whole 16-byte
// residual loads and stores.
#pragma once

#include "epilogue.hpp"
#include "gemm_mx.hpp"

namespace biasact {

namespace mxt {
constexpr int THREADS = 256, STAGES = 3;

template <int SJ, int SI>
struct Tile {
  static constexpr int BM = 64 * SJ, BN = 64 * SI;
  static constexpr int A_STAGE = BM * 64, B_STAGE = BN * 64;
  static constexpr int A_OFF = 0, B_OFF = STAGES * A_STAGE, S_OFF = B_OFF + STAGES * B_STAGE;
  static constexpr int LDS_BYTES = S_OFF + (BM + BN) * 16;       // 78 KB for 256x128: two workgroups a CU
  static constexpr int SLOADS = (BM + BN + THREADS - 1) / THREADS;   // scale rows per thread
  static constexpr int PASS_ROWS = 32 * SJ;
  static_assert(PASS_ROWS * BN * 4 <= LDS_BYTES, "epilogue staging");
};

constexpr int WAIT_LGKM0 = 0xC07F;
constexpr int wait_vm(int n) { return 0x0F70 | (n & 0xF) | ((n >> 4) << 14); }

__device__ __forceinline__ int swz(int row) { return (row >> 2) & 3; }

// 16 bytes per lane from off + soff of the buffer to lds + 16 * lane
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, soff, 0, 0);
}

// acc += b . a^T over 64 k, scale byte KS of each word
template <int KS>
__device__ __forceinline__ f32x16 mfma32(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa) {
  const i32x8 x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const i32x8 y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, KS, (int)sb, KS, (int)sa);
}
}  // namespace mxt

template <int DTO, int SJ, int SI>
__global__ __launch_bounds__(256, 2) void mx_tile_kernel(MxGemmArgs a) {
  using T = mxt::Tile<SJ, SI>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS_BYTES];

  uint32_t tm, tn;
  map_tile(blockIdx.x, gridDim.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t m0 = tm * T::BM, n0 = tn * T::BN;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  const int half = lane >> 5, lrow = lane & 31;
  const int G = (int)a.G;                     // >= 1

  f32x16 acc[SI][SJ];
#pragma unroll
  for (int si = 0; si < SI; ++si)
#pragma unroll
    for (int sj = 0; sj < SJ; ++sj)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[si][sj][r] = 0.0f;

  // ---- direct loads: SJ of A and SI of B per wave and k-tile, 16 rows each --------
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes);
  uint32_t a_off[SJ], b_off[SI];              // rows past the end read as zero
#pragma unroll
  for (int i = 0; i < SJ; ++i) {
    const int row = (SJ * w + i) * 16 + (lane >> 2);
    a_off[i] = m0 + row < a.M ? (m0 + row) * a.G * 64u + ((lane & 3) ^ mxt::swz(row)) * 16u : kOOB;
  }
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int row = (SI * w + i) * 16 + (lane >> 2);
    b_off[i] = n0 + row < a.N ? (n0 + row) * a.G * 64u + ((lane & 3) ^ mxt::swz(row)) * 16u : kOOB;
  }
  auto issue = [&](int kt, int st) {
#pragma unroll
    for (int i = 0; i < SJ; ++i)
      mxt::load_to_lds(ra, smem + T::A_OFF + st * T::A_STAGE + (SJ * w + i) * 1024, a_off[i], kt * 64);
#pragma unroll
    for (int i = 0; i < SI; ++i)
      mxt::load_to_lds(rb, smem + T::B_OFF + st * T::B_STAGE + (SI * w + i) * 1024, b_off[i], kt * 64);
  };

  // ---- scales: thread t brings rows t (and t + 256) of A's rows followed by B's -----
  // words 4 S .. 4 S + 3 of the row, zero from G on (never past the row's own)
  auto load_scales = [&](int S, u32x4 (&v)[T::SLOADS]) {
#pragma unroll
    for (int i = 0; i < T::SLOADS; ++i) {
      const int row0 = i * mxt::THREADS + 64 * w;      // uniform; BM and BN are multiples of 64
      const bool of_a = row0 < T::BM;
      const __amdgpu_buffer_rsrc_t rs = of_a ? make_rsrc(a.As, a.as_bytes) : make_rsrc(a.Bs, a.bs_bytes);
      const uint32_t row = of_a ? m0 + row0 + lane : n0 + (row0 - T::BM) + lane;
      const bool ok = row0 < T::BM + T::BN && row < (of_a ? a.M : a.N);
      const uint32_t at = (row * a.G + 4u * S) * 4u;
      v[i] = u32x4{0, 0, 0, 0};
      if (4 * S + 4 <= G) {
        v[i] = ld_b128(rs, ok ? at : kOOB);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (4 * S + e < G) v[i][e] = ld_b32(rs, ok ? at + e * 4u : kOOB);
      }
    }
  };
  auto put_scales = [&](const u32x4 (&v)[T::SLOADS]) {
#pragma unroll
    for (int i = 0; i < T::SLOADS; ++i)
      if (i * mxt::THREADS + 64 * w < T::BM + T::BN)
        *reinterpret_cast<u32x4*>(smem + T::S_OFF + (i * mxt::THREADS + 64 * w + lane) * 16) = v[i];
  };

  // ---- LDS fragment addresses: row, chunk 2 half + ks ------------------------------
  const int x = mxt::swz(lrow);
  uint32_t a_rd[2], b_rd[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    a_rd[ks] = T::A_OFF + (wm * 32 * SJ + lrow) * 64 + (((2 * half + ks) ^ x) * 16);
    b_rd[ks] = T::B_OFF + (wn * 32 * SI + lrow) * 64 + (((2 * half + ks) ^ x) * 16);
  }

  // ---- main loop ---------------------------------------------------------------------
  // k-tile kt: wait for this wave's loads of it (those of kt + 1 may be in
  // flight), barrier, issue kt + 2 into the stage that kt - 1 held (every wave
  // had its fragments before it came to this barrier), read fragments, multiply.
  constexpr int LOADS = SJ + SI;
  u32x4 snext[T::SLOADS];
  load_scales(0, snext);
  issue(0, 0);
  if (G > 1) issue(1, 1);
  put_scales(snext);
  u32x4 sa[SJ], sb[SI];
  const int sh = 16 * half;
  int st = 0;                                          // kt % 3
  for (int k0 = 0; k0 < G; k0 += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kt = k0 + j;
      if (kt >= G) break;
      if (kt + 1 < G) __builtin_amdgcn_s_waitcnt(mxt::wait_vm(LOADS));
      else __builtin_amdgcn_s_waitcnt(mxt::wait_vm(0));
      __builtin_amdgcn_s_waitcnt(mxt::WAIT_LGKM0);     // the scales this wave put
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const int st2 = st == 0 ? 2 : st - 1;            // (kt + 2) % 3
      if (kt + 2 < G) issue(kt + 2, st2);
      if (j == 0) {
        // every wave put its rows at least one barrier ago; the words stay in
        // registers, and the next four k-tiles' go in from j = 2 on, when every
        // wave has passed the barrier after these reads
#pragma unroll
        for (int sj = 0; sj < SJ; ++sj)
          sa[sj] = *reinterpret_cast<const u32x4*>(smem + T::S_OFF + (wm * 32 * SJ + sj * 32 + lrow) * 16);
#pragma unroll
        for (int si = 0; si < SI; ++si)
          sb[si] = *reinterpret_cast<const u32x4*>(smem + T::S_OFF + (T::BM + wn * 32 * SI + si * 32 + lrow) * 16);
        if (k0 + 4 < G) load_scales((k0 >> 2) + 1, snext);
      }
      if (j == 2 && k0 + 4 < G) put_scales(snext);
      u32x4 fa[SJ][2], fb[SI][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int si = 0; si < SI; ++si)
          fb[si][ks] = *reinterpret_cast<const u32x4*>(smem + b_rd[ks] + st * T::B_STAGE + si * 2048);
#pragma unroll
        for (int sj = 0; sj < SJ; ++sj)
          fa[sj][ks] = *reinterpret_cast<const u32x4*>(smem + a_rd[ks] + st * T::A_STAGE + sj * 2048);
      }
#pragma unroll
      for (int si = 0; si < SI; ++si)
#pragma unroll
        for (int sj = 0; sj < SJ; ++sj)
          acc[si][sj] = mxt::mfma32<0>(fb[si][0], fa[sj][0], acc[si][sj], sb[si][j] >> sh, sa[sj][j] >> sh);
#pragma unroll
      for (int si = 0; si < SI; ++si)
#pragma unroll
        for (int sj = 0; sj < SJ; ++sj)
          acc[si][sj] = mxt::mfma32<1>(fb[si][1], fa[sj][1], acc[si][sj], sb[si][j] >> sh, sa[sj][j] >> sh);
      st = st == 2 ? 0 : st + 1;
    }
  }

  // ---- epilogue -------------------------------------------------------------------
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  constexpr uint32_t ES = Elem<DTO>::bytes;
  constexpr int LPR = T::BN / 8;                       // lanes per row
  // whole 16-byte accesses: rows of a multiple of 8 outputs, aligned bases
  const bool vec = a.N % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R)) & 15u) == 0;
  auto slot = [](int r, int c) { return (uint32_t)(r * (T::BN * 4) + ((c ^ (2 * (r & 15))) << 4)); };
  // this lane's outputs of a row: eight consecutive ones, or columns lane + 64 e
  const int lc = lane % LPR;
  uint32_t idx[8];
  float bv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) idx[e] = vec ? n0 + 8 * lc + e : n0 + lane + 64 * (e % SI);
  load_bias_vec<8>(a.bias, a.bias_bytes, a.bias_dt, idx, a.N, bv);
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    __syncthreads();                                   // the last k-tile, or the previous pass, is read
    if (wm == pass) {
#pragma unroll
      for (int si = 0; si < SI; ++si)
#pragma unroll
        for (int sj = 0; sj < SJ; ++sj)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4*>(smem + slot(sj * 32 + lrow, wn * 8 * SI + si * 8 + 2 * g + half)) =
                f32x4{acc[si][sj][4 * g + 0], acc[si][sj][4 * g + 1], acc[si][sj][4 * g + 2], acc[si][sj][4 * g + 3]};
    }
    __syncthreads();
    const uint32_t mp = m0 + pass * T::PASS_ROWS;
    with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act_c)::value;
      if (vec) {
        with_residual(a.R != nullptr, [&](auto res_c) __attribute__((always_inline)) {
          constexpr bool HAS_R = decltype(res_c)::value;
          constexpr int STEP = mxt::THREADS / LPR;
#pragma unroll 2
          for (int it = 0; it < T::PASS_ROWS / STEP; ++it) {
            const int r = it * STEP + (int)threadIdx.x / LPR;
            const uint32_t m = mp + r, n = n0 + lc * 8;
            const bool ok = m < a.M && n < a.N;
            const uint32_t at = m * a.N + n;
            float z[8], rv[8];
            if constexpr (HAS_R) {
              load4<DTO>(rr, at, ok, *reinterpret_cast<float(*)[4]>(rv));
              load4<DTO>(rr, at + 4, ok, *reinterpret_cast<float(*)[4]>(rv + 4));
            }
            const f32x4 lo = *reinterpret_cast<const f32x4*>(smem + slot(r, 2 * lc));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(smem + slot(r, 2 * lc + 1));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              z[e] = (e < 4 ? lo[e & 3] : hi[e & 3]) + bv[e];
              if constexpr (HAS_R) z[e] += rv[e];
              z[e] = mx::act<ACT, DTO>(z[e], a.alpha);
            }
            if constexpr (ES == 4) {
              store4<DTO>(rc, at, ok, z[0], z[1], z[2], z[3]);
              store4<DTO>(rc, at + 4, ok, z[4], z[5], z[6], z[7]);
            } else {
              u32x4 o;
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = narrow<DTO>(z[2 * e]) | (narrow<DTO>(z[2 * e + 1]) << 16);
              st_b128(rc, ok ? at * ES : kOOB, o);
            }
          }
        });
      } else {
        for (int it = 0; it < T::PASS_ROWS / 4; ++it) {
          const int r = it * 4 + w;
          const uint32_t m = mp + r;
#pragma unroll
          for (int e = 0; e < SI; ++e) {
            const int c = lane + 64 * e;
            const bool ok = m < a.M && n0 + c < a.N;
            const uint32_t at = m * a.N + n0 + c;
            float z = *reinterpret_cast<const float*>(smem + slot(r, c >> 2) + (c & 3) * 4) + bv[e];
            if (a.R) z += load1<DTO>(rr, at, ok);
            store1<DTO>(rc, at, ok, mx::act<ACT, DTO>(z, a.alpha));
          }
        }
      }
    });
  }
}

template <int DTO, int SJ, int SI>
inline void launch_mx_tile(MxGemmArgs a, hipStream_t s) {
  using T = mxt::Tile<SJ, SI>;
  a.tiles_n = (a.N + T::BN - 1) / T::BN;
  a.tiles_m = (a.M + T::BM - 1) / T::BM;
  note_launch("gemm mxfp4 tile, %d m x %d n", T::BM, T::BN);
  launch_kernel(mx_tile_kernel<DTO, SJ, SI>, dim3(a.tiles_m * a.tiles_n), dim3(mxt::THREADS), s, a);
}

}  // namespace biasact
