// tile_epilogue.hpp — bias, residual, activation and stores of a workgroup's
// tile of sums that its waves hold as 32x32 accumulator blocks.
//
// Every wave works by itself: 32 rows at a time, each lane adds the bias, applies
// the activation to its own sums and puts the rounded values into LDS of the
// wave's own (rows 16 bytes apart beyond their length, which spreads a column's
// accesses over the banks), from where it stores pieces of whole cache lines, 16
// bytes a lane.  A residual comes in the same way, its loads 32 rows ahead.  No barrier
// holds up one wave's stores for another's arithmetic.  The sums before the
// activation (Z) leave by a round of their own before C's.
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

// acc[si][sj][e] of lane (half, lrow) of wave (wm, wn): the sum of
//   m = m0 + 32 (SJ wm + sj) + lrow,  n = n0 + 32 (SI wn + si) + 8 (e / 4) + 4 half + e % 4.
// smem: 32 rows of each wave's columns from 0 on, this tile's bias as floats at
// bias_off behind them.  Args: M, N, C, Z, R, c_bytes, act and alpha of the call.
template <int DTO, int WM, int WN, int SJ, int SI, class Args>
__device__ __forceinline__ void tile_epilogue(const Args& a, uint8_t* smem, uint32_t bias_off, uint32_t m0, uint32_t n0,
                                              f32x16 (&acc)[SI][SJ]) {
  constexpr int ES = Elem<DTO>::bytes, EPC = 16 / ES;  // bytes an output, outputs a chunk
  constexpr int COLS = 32 * SI, CPR = COLS / EPC;      // a wave's columns; chunks, and lanes, a row
  constexpr int PITCH = COLS * ES + 16, RPI = 64 / CPR, CHUNKS = 32 / RPI;   // rows an instruction covers
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w / WN, wn = w % WN;
  // The lane's number, told to the compiler anew: addresses computed from it
  // here would otherwise be kept in registers through the main loop.
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int row = lane & 31, four = 4 * (lane >> 5);
  const uint32_t m_wave = m0 + 32 * SJ * wm, n_wave = n0 + COLS * wn;
  uint8_t* const mine = smem + w * (32 * PITCH);
  const float* const bias = reinterpret_cast<const float*>(smem + bias_off) + COLS * wn;
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  // whole 16-byte accesses: rows of whole chunks, aligned bases
  const bool vec = a.N % EPC == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R) |
                                       reinterpret_cast<uintptr_t>(a.Z)) & 15u) == 0;
  // f(i, LDS address, byte offset in C or kOOB) for every chunk of 32 rows
  const int crow = lane / CPR, cc = lane % CPR;
  const bool n_ok = n_wave + cc * EPC < a.N;
  auto by_chunk = [&](int sj, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int r = i * RPI + crow;
      const uint32_t m = m_wave + 32 * sj + r;
      f(i, mine + r * PITCH + cc * 16, n_ok && m < a.M ? (m * a.N + n_wave + cc * EPC) * ES : kOOB);
    }
  };
  // the same for every single output, four rows at a time from row `from` on
  constexpr int E = COLS / 64 > 0 ? COLS / 64 : 1;
  auto by_output = [&](int sj, int from, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4 * E; ++i) {
      const int r = from + i / E, c = lane + 64 * (i % E);
      const uint32_t m = m_wave + 32 * sj + r;
      f(i, mine + r * PITCH + c * ES, m < a.M && n_wave + c < a.N ? (m * a.N + n_wave + c) * ES : kOOB);
    }
  };
  static_assert(COLS % 64 == 0, "by_output");
  u32x4 res[CHUNKS];                                   // the next 32 rows' residual
  auto load_res = [&](int sj) __attribute__((always_inline)) {
    by_chunk(sj, [&](int i, uint8_t*, uint32_t at) { res[i] = tep::load_once(rr, at); });
  };
  if (a.R && vec) load_res(0);
  __syncthreads();                                     // the last k-step is read by every wave
#pragma unroll 1
  for (int out = a.Z ? 0 : 1; out < 2; ++out) {
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(out ? a.C : a.Z, a.c_bytes);
    auto rows = [&](auto sj_c) __attribute__((always_inline)) {
      constexpr int sj = decltype(sj_c)::value;
      if (a.R) {
        if (vec) {
          by_chunk(sj, [&](int i, uint8_t* p, uint32_t) { *reinterpret_cast<u32x4*>(p) = res[i]; });
          if (sj + 1 < SJ || out == 0) load_res((sj + 1) % SJ);
        } else {
#pragma unroll 1
          for (int from = 0; from < 32; from += 4) {
            uint32_t v[4 * E];
            by_output(sj, from, [&](int i, uint8_t*, uint32_t at) {
              if constexpr (ES == 4) v[i] = ld_b32(rr, at);
              else v[i] = ld_b16(rr, at);
            });
            by_output(sj, from, [&](int i, uint8_t* p, uint32_t) {
              if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(p) = v[i];
              else *reinterpret_cast<uint16_t*>(p) = (uint16_t)v[i];
            });
          }
        }
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
      if (vec) {
        by_chunk(sj, [&](int, uint8_t* p, uint32_t at) { tep::store_once(rc, at, *reinterpret_cast<const u32x4*>(p)); });
      } else {
#pragma unroll 1
        for (int from = 0; from < 32; from += 4)
          by_output(sj, from, [&](int, uint8_t* p, uint32_t at) {
            if constexpr (ES == 4) st_b32(rc, at, *reinterpret_cast<const uint32_t*>(p));
            else st_b16(rc, at, *reinterpret_cast<const uint16_t*>(p));
          });
      }
      tep::lds_order();
    };
    rows(std::integral_constant<int, 0>{});
    rows(std::integral_constant<int, 1>{});
    if constexpr (SJ > 2) {
      rows(std::integral_constant<int, 2>{});
      rows(std::integral_constant<int, 3>{});
    }
  }
}

}  // namespace biasact
