// gemm_mx_tile.hpp — large-tile fused product of two MXFP4 operands on gfx950:
//   C[M,N] = act(A . B^T + bias (+ R)), both operands as rows of k (mx_args.hpp)
//
// Workgroup: 512 threads = 8 waves, output tile 256 (m) x 256 (n), k-tile of
// one group of 128 values (64 bytes of codes and 4 scale bytes a row).  Waves
// 0-3 form cluster 0, waves 4-7 cluster 1; wave w owns the 128 (m) x 64 (n)
// sub-tile at m = 128 (w / 4), n = 64 (w % 4): 4 x 2 accumulator blocks of
// 32x32.  The clusters alternate phases between workgroup barriers (one wave
// of each on every SIMD): while one multiplies a k-tile from registers, 16
// v_mfma_scale_f32_32x32x64, the other reads its fragments of the next one from
// LDS and issues its global loads of the k-tile three ahead.
//
// Codes reach LDS without passing through registers, 16 bytes a lane; four
// stages of A and B, chunk c of row r at slot c ^ ((r >> 2) & 3), so the eight
// lanes that a 16-byte LDS read serves at a time are on different banks.  Half
// h of a wave takes chunks 2 h and 2 h + 1 of its rows: its two scale bytes
// are then neighbours, and one shift puts them where the instruction's operand
// selector reads byte 0 for the first k-step and byte 1 for the second.
// Scales travel 16 bytes a row for four k-tiles at once (one load per wave):
// fetched with each k-tile they would touch one cache line per row and tile,
// as many as the codes do.
//
// Epilogue: the fp32 sums leave through LDS in two passes of 128 rows (chunk c
// of a 1 KB row at slot c ^ 2 (r & 31)), so every lane handles eight
// consecutive outputs of a row: one bias fetch for all its rows, whole 16-byte
// residual loads and stores.
#pragma once

#include "epilogue.hpp"
#include "gemm_mx.hpp"

namespace biasact {

namespace mxt {
constexpr int BM = 256, BN = 256, THREADS = 512, STAGES = 4;
constexpr int STAGE = 256 * 64;                            // one operand's k-tile
constexpr int A_OFF = 0, B_OFF = STAGES * STAGE, S_OFF = 2 * STAGES * STAGE;
constexpr int S_BUF = 512 * 16;                            // scales of 256 + 256 rows for four k-tiles
constexpr int LDS_BYTES = S_OFF + 2 * S_BUF;               // 144 KB
constexpr int LOADS = 4;                                   // direct loads per wave per k-tile

constexpr int WAIT_LGKM0 = 0xC07F;
constexpr int wait_vm(int n) { return 0x0F70 | (n & 0xF) | ((n >> 4) << 14); }

__device__ __forceinline__ int swz(int row) { return (row >> 2) & 3; }

// acc += b . a^T over 64 k, scale byte KS of each word
template <int KS>
__device__ __forceinline__ f32x16 mfma32(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa) {
  const i32x8 x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const i32x8 y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, KS, (int)sb, KS, (int)sa);
}
}  // namespace mxt

template <int DTO>
__global__ __launch_bounds__(512, 1) void mx_tile_kernel(MxGemmArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[mxt::LDS_BYTES];

  uint32_t tm, tn;
  map_tile(blockIdx.x, gridDim.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t m0 = tm * mxt::BM, n0 = tn * mxt::BN;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 2, wn = w & 3;          // cluster == wm
  const int half = lane >> 5, lrow = lane & 31;
  const int G = (int)a.G;

  f32x16 acc[2][4];
#pragma unroll
  for (int si = 0; si < 2; ++si)
#pragma unroll
    for (int sj = 0; sj < 4; ++sj)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[si][sj][r] = 0.0f;

  // ---- direct loads: instruction i covers stage rows (2 w + i) * 16 .. + 16 ----
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, a.a_bytes);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, a.b_bytes);
  uint32_t a_off[2], b_off[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (2 * w + i) * 16 + (lane >> 2);
    const uint32_t c = (lane & 3) ^ mxt::swz(row);
    a_off[i] = m0 + row < a.M ? (m0 + row) * a.G * 64u + c * 16u : kOOB;     // rows past the end read as zero
    b_off[i] = n0 + row < a.N ? (n0 + row) * a.G * 64u + c * 16u : kOOB;
  }
  // One direct load j (0..3) of k-tile kt into stage st.  A k-tile past the
  // last repeats that one (into a stage that nobody reads any more).
  auto issue_one = [&](int kt, int st, int j) {
    const int i = j >> 1;
    const int so = min(kt, G - 1) * 64;
    if ((j & 1) == 0)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ra, (lds_void*)(smem + mxt::A_OFF + st * mxt::STAGE + (2 * w + i) * 1024), 16, a_off[i], so, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_void*)(smem + mxt::B_OFF + st * mxt::STAGE + (2 * w + i) * 1024), 16, b_off[i], so, 0, 0);
  };

  // ---- scales: lane l of wave w brings row 64 w + l (A's rows, then B's) --------
  const __amdgpu_buffer_rsrc_t rs = w < 4 ? make_rsrc(a.As, a.as_bytes) : make_rsrc(a.Bs, a.bs_bytes);
  const uint32_t srow = w < 4 ? m0 + 64 * w + lane : n0 + 64 * (w - 4) + lane;
  const uint32_t s_off = srow < (w < 4 ? a.M : a.N) ? srow * a.G * 4u : kOOB;
  // words 4 S .. 4 S + 3 of the row, zero from G on (never past the row's own)
  auto load_scales = [&](int S) {
    u32x4 v = {0, 0, 0, 0};
    if (4 * S + 4 <= G) {
      v = ld_b128(rs, s_off == kOOB ? kOOB : s_off + S * 16u);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (4 * S + e < G) v[e] = ld_b32(rs, s_off == kOOB ? kOOB : s_off + S * 16u + e * 4u);
    }
    return v;
  };
  auto store_scales = [&](int S, u32x4 v) {
    *reinterpret_cast<u32x4*>(smem + mxt::S_OFF + (S & 1) * mxt::S_BUF + (64 * w + lane) * 16) = v;
  };

  // ---- LDS fragment addresses: row, chunk 2 half + ks ---------------------------
  const int x = mxt::swz(lrow);
  uint32_t a_rd[2], b_rd[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    a_rd[ks] = mxt::A_OFF + (wm * 128 + lrow) * 64 + (((2 * half + ks) ^ x) * 16);
    b_rd[ks] = mxt::B_OFF + (wn * 64 + lrow) * 64 + (((2 * half + ks) ^ x) * 16);
  }

  // ---- prologue: scales of k-tiles 0 .. 3, k-tiles 0 .. 2 in flight, 0 landed ----
  if (G > 0) {
    store_scales(0, load_scales(0));
    for (int t = 0; t < mxt::STAGES - 1; ++t)
#pragma unroll
      for (int j = 0; j < mxt::LOADS; ++j) issue_one(t, t, j);
    __builtin_amdgcn_s_waitcnt(mxt::wait_vm(2 * mxt::LOADS));
    __builtin_amdgcn_s_waitcnt(mxt::WAIT_LGKM0);
  }
  __builtin_amdgcn_s_barrier();
  if (wm == 1) __builtin_amdgcn_s_barrier();      // cluster 1 runs one phase behind

  // Intervals as between barriers: cluster 0 reads k-tile t at 2 t and
  // multiplies it at 2 t + 1, cluster 1 one later.  Reading t also loads
  // k-tile t + 3 into stage (t + 3) % 4 = (t - 1) % 4, whose last reader ended
  // by interval 2 t - 1, and waits for its own loads of t + 1 before the
  // barrier that precedes their first read at interval 2 t + 2.
  u32x4 fa[4][2], fb[2][2];
  u32x4 sa[4], sb[2], snext = {0, 0, 0, 0};
  const int sh = 16 * half;
  for (int k0 = 0; k0 < G; k0 += 4) {
    const int S = k0 >> 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kt = k0 + j;
      if (kt >= G) break;
      // ---- memory phase --------------------------------------------------------
      __builtin_amdgcn_sched_barrier(0);
      if (j == 0) {
        if (k0 + 4 < G) snext = load_scales(S + 1);
        const uint8_t* sp = smem + mxt::S_OFF + (S & 1) * mxt::S_BUF;
#pragma unroll
        for (int sj = 0; sj < 4; ++sj)
          sa[sj] = *reinterpret_cast<const u32x4*>(sp + (wm * 128 + sj * 32 + lrow) * 16);
#pragma unroll
        for (int si = 0; si < 2; ++si)
          sb[si] = *reinterpret_cast<const u32x4*>(sp + (256 + wn * 64 + si * 32 + lrow) * 16);
      }
      // the other buffer's last readers passed at least two barriers ago
      if (j == 2 && k0 + 4 < G) store_scales(S + 1, snext);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int sj = 0; sj < 4; ++sj) {
          fa[sj][ks] = *reinterpret_cast<const u32x4*>(smem + a_rd[ks] + j * mxt::STAGE + sj * 2048);
          if (sj & 1) {              // one direct load after every second A fragment
            __builtin_amdgcn_sched_barrier(0);
            issue_one(kt + 3, (j + 3) & 3, ks * 2 + (sj >> 1));
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int si = 0; si < 2; ++si)
          fb[si][ks] = *reinterpret_cast<const u32x4*>(smem + b_rd[ks] + j * mxt::STAGE + si * 2048);
      }
      // k-tile kt + 1 landed for this wave (kt + 2, kt + 3 and at j = 0 the
      // scales between them may be in flight)
      if (j == 0) __builtin_amdgcn_s_waitcnt(mxt::wait_vm(2 * mxt::LOADS + 1));
      else __builtin_amdgcn_s_waitcnt(mxt::wait_vm(2 * mxt::LOADS));
      __builtin_amdgcn_s_waitcnt(mxt::WAIT_LGKM0);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // ---- compute phase: 16 matrix instructions from registers -----------------
#pragma unroll
      for (int si = 0; si < 2; ++si)
#pragma unroll
        for (int sj = 0; sj < 4; ++sj)
          acc[si][sj] = mxt::mfma32<0>(fb[si][0], fa[sj][0], acc[si][sj], sb[si][j] >> sh, sa[sj][j] >> sh);
#pragma unroll
      for (int si = 0; si < 2; ++si)
#pragma unroll
        for (int sj = 0; sj < 4; ++sj)
          acc[si][sj] = mxt::mfma32<1>(fb[si][1], fa[sj][1], acc[si][sj], sb[si][j] >> sh, sa[sj][j] >> sh);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
    }
  }
  // no direct load may still be writing LDS when the epilogue reuses it
  __builtin_amdgcn_s_waitcnt(mxt::wait_vm(0));
  if (wm == 0) __builtin_amdgcn_s_barrier();      // same barrier count for both clusters

  // ---- epilogue -------------------------------------------------------------------
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  constexpr uint32_t ES = Elem<DTO>::bytes;
  // whole 16-byte accesses: rows of a multiple of 8 outputs, aligned bases
  const bool vec = a.N % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R)) & 15u) == 0;
  auto slot = [](int r, int c) { return (uint32_t)(r * 1024 + ((c ^ (2 * (r & 31))) << 4)); };
  // this lane's outputs of a row: eight consecutive ones, or columns lane + 64 e
  uint32_t idx[8];
  float bv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) idx[e] = vec ? n0 + 8 * lrow + e : n0 + lane + 64 * (e & 3);
  load_bias_vec<8>(a.bias, a.bias_bytes, a.bias_dt, idx, a.N, bv);
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    __syncthreads();
    if (wm == pass) {
#pragma unroll
      for (int si = 0; si < 2; ++si)
#pragma unroll
        for (int sj = 0; sj < 4; ++sj)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4*>(smem + slot(sj * 32 + lrow, wn * 16 + si * 8 + 2 * g + half)) =
                f32x4{acc[si][sj][4 * g + 0], acc[si][sj][4 * g + 1], acc[si][sj][4 * g + 2], acc[si][sj][4 * g + 3]};
    }
    __syncthreads();
    with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act_c)::value;
      if (vec) {
        with_residual(a.R != nullptr, [&](auto res_c) __attribute__((always_inline)) {
          constexpr bool HAS_R = decltype(res_c)::value;
#pragma unroll 2
          for (int it = 0; it < 8; ++it) {
            const int r = it * 16 + 2 * w + half;
            const uint32_t m = m0 + pass * 128 + r, n = n0 + lrow * 8;
            const bool ok = m < a.M && n < a.N;
            const uint32_t at = m * a.N + n;
            float z[8], rv[8];
            if constexpr (HAS_R) {
              load4<DTO>(rr, at, ok, *reinterpret_cast<float(*)[4]>(rv));
              load4<DTO>(rr, at + 4, ok, *reinterpret_cast<float(*)[4]>(rv + 4));
            }
            const f32x4 lo = *reinterpret_cast<const f32x4*>(smem + slot(r, 2 * lrow));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(smem + slot(r, 2 * lrow + 1));
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
        for (int it = 0; it < 16; ++it) {
          const int r = it * 8 + w;
          const uint32_t m = m0 + pass * 128 + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
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

template <int DTO>
inline void launch_mx_tile(MxGemmArgs a, hipStream_t s) {
  a.tiles_n = (a.N + mxt::BN - 1) / mxt::BN;
  a.tiles_m = (a.M + mxt::BM - 1) / mxt::BM;
  note_launch("gemm mxfp4 256x256 ping-pong");
  launch_kernel(mx_tile_kernel<DTO>, dim3(a.tiles_m * a.tiles_n), dim3(mxt::THREADS), s, a);
}

}  // namespace biasact
