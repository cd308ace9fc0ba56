// tile_epilogue.hpp — bias, residual, activation and stores of a workgroup's
// tile of sums that its waves hold as 32x32 accumulator blocks.
//
// Each lane adds the bias, applies the activation to its own sums and puts the
// rounded values into LDS (16-byte chunk c of row r at slot c ^ r, within the
// row), from where whole rows are stored, 16 bytes a lane.  A residual comes in
// the same way: whole rows into LDS, then each value to the lane that holds its
// sum.  16-bit outputs take one pass, 32-bit ones a pass for each wm.  The
// sums before the activation (Z) leave by a round of their own before C's.
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
// smem: room for the pass's rows from 0 on, this tile's bias as floats at
// bias_off behind them.  Args: M, N, C, Z, R, c_bytes, act and alpha of the call.
template <int DTO, int WM, int WN, int SJ, int SI, class Args>
__device__ __forceinline__ void tile_epilogue(const Args& a, uint8_t* smem, uint32_t bias_off, uint32_t m0, uint32_t n0,
                                              f32x16 (&acc)[SI][SJ]) {
  constexpr int THREADS = 64 * WM * WN, BM = 32 * SJ * WM, BN = 32 * SI * WN;
  constexpr int ES = Elem<DTO>::bytes, EPC = 16 / ES;  // bytes an output, outputs a chunk
  constexpr int CPR = BN / EPC;                        // chunks, and lanes, a row
  constexpr int PASSES = ES == 2 ? 1 : WM, ROWS = BM / PASSES;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w / WN, wn = w % WN;
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  // whole 16-byte accesses: rows of whole chunks, aligned bases
  const bool vec = a.N % EPC == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R) |
                                       reinterpret_cast<uintptr_t>(a.Z)) & 15u) == 0;
  // The thread's number, told to the compiler anew: addresses computed from it
  // here would otherwise be kept in registers through the main loop.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  auto slot = [](int r, int c) { return (uint32_t)(r * (BN * ES) + ((c ^ (r & (CPR - 1))) << 4)); };
  // f(LDS address, element offset in C, whether there is such an output), for
  // every chunk of the pass's rows, a row's chunks in neighbouring lanes
  constexpr int CHUNKS = ROWS * CPR / THREADS;
  auto by_chunk = [&](int pass, int from, int count, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < count; ++i) {
      const int r = (from + i) * (THREADS / CPR) + tid / CPR, c = tid % CPR;
      const uint32_t m = m0 + pass * ROWS + r, n = n0 + c * EPC;
      f(i, slot(r, c), m * a.N + n, m < a.M && n < a.N);
    }
  };
  // the same for every single output, a wave's 64 E of count rows at a time
  constexpr int E = BN / 64;
  auto by_output = [&](int pass, int from, int count, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < count * E; ++i) {
      const int r = (from + i / E) * (WM * WN) + w, c = (tid & 63) + 64 * (i % E);
      const uint32_t m = m0 + pass * ROWS + r, n = n0 + c;
      f(i, slot(r, c / EPC) + (c % EPC) * ES, m * a.N + n, m < a.M && n < a.N);
    }
  };
#pragma unroll 1
  for (int round = a.Z ? 0 : PASSES; round < 2 * PASSES; ++round) {
    const bool to_z = round < PASSES;                  // uniform
    const int pass = to_z ? round : round - PASSES;
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(to_z ? a.Z : a.C, a.c_bytes);
    asm volatile("" : "+v"(tid));
    const int row = tid & 31, four = 4 * ((tid >> 5) & 1);
    __syncthreads();                                   // the last k-step, or the previous pass, is read
    if (a.R) {
      // eight or more loads at a time: a write to LDS waits for all earlier loads
      if (vec) {
#pragma unroll 1
        for (int from = 0; from < CHUNKS; from += 8) {
          u32x4 v[8];
          by_chunk(pass, from, 8, [&](int i, uint32_t, uint32_t at, bool ok) { v[i] = tep::load_once(rr, ok ? at * ES : kOOB); });
          by_chunk(pass, from, 8, [&](int i, uint32_t p, uint32_t, bool) { *reinterpret_cast<u32x4*>(smem + p) = v[i]; });
        }
      } else {
#pragma unroll 1
        for (int from = 0; from < ROWS / (WM * WN); from += 4) {
          uint32_t v[4 * E];
          by_output(pass, from, 4, [&](int i, uint32_t, uint32_t at, bool ok) {
            if constexpr (ES == 4) v[i] = ld_b32(rr, ok ? at * ES : kOOB);
            else v[i] = ld_b16(rr, ok ? at * ES : kOOB);
          });
          by_output(pass, from, 4, [&](int i, uint32_t p, uint32_t, bool) {
            if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(smem + p) = v[i];
            else *reinterpret_cast<uint16_t*>(smem + p) = (uint16_t)v[i];
          });
        }
      }
      __syncthreads();
    }
    if (PASSES == 1 || wm == pass) {
      with_act(to_z ? ACT_NONE : a.act, [&](auto act_c) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act_c)::value;
        with_residual(a.R != nullptr, [&](auto res_c) __attribute__((always_inline)) {
#pragma unroll
          for (int si = 0; si < SI; ++si)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int n = (wn * SI + si) * 32 + 8 * g + four;
              const f32x4 bias = *reinterpret_cast<const f32x4*>(smem + bias_off + n * 4);
#pragma unroll
              for (int sj = 0; sj < SJ; ++sj) {
                // four consecutive outputs; no other lane touches them.  One group at
                // a time: there are few registers beside the sums.
                __builtin_amdgcn_sched_barrier(0);
                const int r = (PASSES == 1 ? wm * 32 * SJ : 0) + sj * 32 + row;
                uint8_t* p = smem + slot(r, n / EPC) + (n % EPC) * ES;
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = acc[si][sj][4 * g + e] + bias[e];
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
            }
        });
      });
    }
    __syncthreads();
    if (vec) {
#pragma unroll 1
      for (int from = 0; from < CHUNKS; from += 8)
        by_chunk(pass, from, 8, [&](int, uint32_t p, uint32_t at, bool ok) {
          tep::store_once(rc, ok ? at * ES : kOOB, *reinterpret_cast<const u32x4*>(smem + p));
        });
    } else {
#pragma unroll 1
      for (int from = 0; from < ROWS / (WM * WN); from += 4)
        by_output(pass, from, 4, [&](int, uint32_t p, uint32_t at, bool ok) {
          if constexpr (ES == 4) st_b32(rc, ok ? at * ES : kOOB, *reinterpret_cast<const uint32_t*>(smem + p));
          else st_b16(rc, ok ? at * ES : kOOB, *reinterpret_cast<const uint16_t*>(smem + p));
        });
    }
  }
}

}  // namespace biasact
