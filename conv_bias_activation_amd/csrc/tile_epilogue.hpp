// tile_epilogue.hpp — bias, residual, activation and stores of a workgroup's
// tile of sums that its waves hold as 32x32 accumulator blocks.
//
// Every wave works by itself: 32 rows at a time, each lane adds the bias, applies
// the activation to its own sums and puts the rounded values into LDS of the
// wave's own (rows 16 bytes apart beyond their length, which spreads a column's
// accesses over the banks), from where it stores pieces of whole cache lines, 16
// bytes a lane.  A residual comes in the same way, its loads 32 rows ahead.  No barrier
// holds up one wave's stores for another's arithmetic.  The sums before the
// activation (Z) leave by a round of their own before C's, which reads the residual
// again.  4096^3 bf16, us in a trace: 57, with GELU and Z 67, with a residual 70, with
// GELU, Z and a residual 94 (each of Z and R is 33.6 MB, 6.8 us at a large copy's rate).  With two barriers for every 32
// rows instead, 4096^3 with GELU took 63.2 us (61.7) and 32768x4096x1024 158 (154).
#pragma once

#include "epilogue.hpp"
#include "mx_act.hpp"

namespace biasact {
namespace tep {

// 16 bytes that a kernel touches once (cache policy "non-temporal")
__device__ __forceinline__ u32x4 load_once(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2);
}
__device__ __forceinline__ void store_once(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);
}

// Orders a wave's LDS accesses before and after (the hardware runs them in
// order; this keeps the compiler from exchanging them).
__device__ __forceinline__ void lds_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// narrow<DTO> of two values into one word, by one instruction
template <int DTO>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (DTO == DT_F16) {
    asm("" : "+v"(lo), "+v"(hi));                      // as in narrow: fp32 first
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), f16x2));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
  }
}

}  // namespace tep

// acc[si][sj][e] of lane (half, lrow): the sum of
//   m = m_wave + 32 sj + lrow,  n = n_wave + 32 si + 8 (e / 4) + 4 half + e % 4.
// smem: 32 rows of the columns of each wave w of the workgroup from 0 on, this tile's
// bias as floats at bias_off behind them, the wave's from column 32 SI wn on.  Args: M, N, C, Z, R, c_bytes, act and alpha of the call.
template <int DTO, int SJ, int SI, class Args>
__device__ __forceinline__ void tile_epilogue(const Args& a, uint8_t* smem, uint32_t bias_off, int w, uint32_t m_wave,
                                              uint32_t n_wave, int wn, f32x16 (&acc)[SI][SJ]) {
  constexpr int ES = Elem<DTO>::bytes, EPC = 16 / ES;  // bytes an output, outputs a chunk
  constexpr int COLS = 32 * SI, CPR = COLS / EPC;      // a wave's columns; chunks, and lanes, a row
  constexpr int PITCH = COLS * ES + 16, RPI = 64 / CPR, CHUNKS = 32 / RPI;   // rows an instruction covers
  // The lane's number, told to the compiler anew: addresses computed from it
  // here would otherwise be kept in registers through the main loop.
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int row = lane & 31, four = 4 * (lane >> 5);
  uint8_t* const mine = smem + w * (32 * PITCH);
  const float* const bias = reinterpret_cast<const float*>(smem + bias_off) + COLS * wn;
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  // f(i, LDS address, byte offset in C or kOOB, outputs of the chunk within the row)
  // for every chunk of 32 rows.  A chunk need only be aligned for one output (the
  // GPU runs with unaligned access on); one that the row's end cuts goes output by
  // output.
  const int crow = lane / CPR, cc = lane % CPR;
  const uint32_t n_chunk = n_wave + cc * EPC, inside = n_chunk < a.N ? min(a.N - n_chunk, (uint32_t)EPC) : 0u;
  const bool ragged = __any(inside != (uint32_t)EPC);  // uniform
  auto by_chunk = [&](int sj, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int r = i * RPI + crow;
      const uint32_t m = m_wave + 32 * sj + r;
      f(i, mine + r * PITCH + cc * 16, m < a.M ? (m * a.N + n_chunk) * ES : kOOB);
    }
  };
  u32x4 res[CHUNKS];                                   // the next 32 rows' residual
  auto load_res = [&](int sj) __attribute__((always_inline)) {
    by_chunk(sj, [&](int i, uint8_t*, uint32_t at) {
      res[i] = tep::load_once(rr, inside == (uint32_t)EPC ? at : kOOB);
    });
    if (ragged)
      by_chunk(sj, [&](int i, uint8_t*, uint32_t at) {
        if (inside == (uint32_t)EPC || at == kOOB) return;
#pragma unroll
        for (uint32_t e = 0; e < (uint32_t)EPC; ++e)
          if (e < inside) {
            if constexpr (ES == 4) res[i][e] = ld_b32(rr, at + 4u * e);
            else res[i][e >> 1] |= (uint32_t)ld_b16(rr, at + 2u * e) << (16 * (e & 1));
          }
      });
  };
  if (a.R) load_res(0);
  __syncthreads();                                     // the last k-step is read by every wave
#pragma unroll 1
  for (int out = a.Z ? 0 : 1; out < 2; ++out) {
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(out ? a.C : a.Z, a.c_bytes);
    auto rows = [&](auto sj_c) __attribute__((always_inline)) {
      constexpr int sj = decltype(sj_c)::value;
      if (a.R) {
        by_chunk(sj, [&](int i, uint8_t* p, uint32_t) { *reinterpret_cast<u32x4*>(p) = res[i]; });
        if (sj + 1 < SJ || out == 0) load_res((sj + 1) % SJ);
        tep::lds_order();
      }
      with_act(out ? a.act : ACT_NONE, [&](auto act_c) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act_c)::value;
        with_residual(a.R != nullptr, [&](auto res_c) __attribute__((always_inline)) {
#pragma unroll
          for (int si = 0; si < SI; ++si)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              // four consecutive outputs.  One group at a time: there are few
              // registers beside the sums.
              __builtin_amdgcn_sched_barrier(0);
              const int n = si * 32 + 8 * g + four;
              const f32x4 b = *reinterpret_cast<const f32x4*>(bias + n);
              uint8_t* const p = mine + row * PITCH + n * ES;
              float z[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) z[e] = acc[si][sj][4 * g + e] + b[e];
              if constexpr (ES == 2) {
                if constexpr (decltype(res_c)::value) {
                  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
                  for (int e = 0; e < 4; ++e) z[e] += widen<DTO>((v[e >> 1] >> (16 * (e & 1))) & 0xffffu);
                }
                u32x2 o;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  o[e] = tep::narrow2<DTO>(mx::act<ACT, DTO>(z[2 * e], a.alpha), mx::act<ACT, DTO>(z[2 * e + 1], a.alpha));
                *reinterpret_cast<u32x2*>(p) = o;
              } else {
                if constexpr (decltype(res_c)::value) {
                  const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
                  for (int e = 0; e < 4; ++e) z[e] += v[e];
                }
                f32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = mx::act<ACT, DTO>(z[e], a.alpha);
                *reinterpret_cast<f32x4*>(p) = o;
              }
            }
        });
      });
      tep::lds_order();
      by_chunk(sj, [&](int, uint8_t* p, uint32_t at) {
        tep::store_once(rc, inside == (uint32_t)EPC ? at : kOOB, *reinterpret_cast<const u32x4*>(p));
      });
      if (ragged)
        by_chunk(sj, [&](int, uint8_t* p, uint32_t at) {
          if (inside == (uint32_t)EPC || at == kOOB) return;
#pragma unroll
          for (uint32_t e = 0; e < (uint32_t)EPC; ++e)
            if (e < inside) {
              if constexpr (ES == 4) st_b32(rc, at + 4u * e, *reinterpret_cast<const uint32_t*>(p + 4 * e));
              else st_b16(rc, at + 2u * e, *reinterpret_cast<const uint16_t*>(p + 2 * e));
            }
        });
      tep::lds_order();
    };
    rows(std::integral_constant<int, 0>{});
    if constexpr (SJ > 1) rows(std::integral_constant<int, 1>{});
    if constexpr (SJ > 2) {
      rows(std::integral_constant<int, 2>{});
      rows(std::integral_constant<int, 3>{});
    }
  }
}

// The same for a small tile whose sums lie in LDS as VERSIONS parts [BM][BN] of
// rows 4 floats apart beyond their length, added in order: a thread takes quads of
// four consecutive n.  load() brings bias and residual, and may run early.
template <int DTO, int BM, int BN, int VERSIONS, int THREADS>
struct SumEpilogue {
  static constexpr int QUADS = BM * BN / 4, P = (QUADS + THREADS - 1) / THREADS;
  static constexpr int LDR = BN + 4, SUMS = BM * LDR * 4;
  float add[P][4];
  uint32_t at[P];                                      // element offset of the quad, or kOOB

  template <class Args>
  __device__ __forceinline__ void load(const Args& a, uint32_t m0, uint32_t n0) {
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t o = threadIdx.x + THREADS * p, ml = o / (BN / 4), nl = (o - ml * (BN / 4)) * 4;
      const uint32_t m = m0 + ml, n = n0 + nl;
      const bool in = o < (uint32_t)QUADS && m < a.M && n < a.N;
      at[p] = in ? m * a.N + n : kOOB;
      uint32_t idx[4] = {n, n + 1, n + 2, n + 3};
      load_bias_vec<4>(a.bias, a.bias_bytes, a.bias_dt, idx, in ? a.N : 0u, add[p]);
      if (a.R) {
        float rv[4];
        if (n + 4 <= a.N) {                            // (of any alignment)
          load4<DTO>(rr, at[p], in, rv);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) rv[e] = load1<DTO>(rr, at[p] + e, in && n + e < a.N);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) add[p][e] += rv[e];
      }
    }
  }

  template <class Args>
  __device__ __forceinline__ void store(const Args& a, const uint8_t* smem, uint32_t n0) {
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes), rz = make_rsrc(a.Z, a.Z ? a.c_bytes : 0u);
    with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act_c)::value;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (at[p] == kOOB) continue;
        const uint32_t o = threadIdx.x + THREADS * p, ml = o / (BN / 4), nl = (o - ml * (BN / 4)) * 4;
        const uint8_t* const s = smem + (ml * LDR + nl) * 4u;
        f32x4 z = *reinterpret_cast<const f32x4*>(s);
#pragma unroll
        for (int v = 1; v < VERSIONS; ++v) z += *reinterpret_cast<const f32x4*>(s + v * SUMS);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[e] += add[p][e];
          y[e] = mx::act<ACT, DTO>(z[e], a.alpha);
        }
        if (n0 + nl + 4 <= a.N) {
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
};

}  // namespace biasact
