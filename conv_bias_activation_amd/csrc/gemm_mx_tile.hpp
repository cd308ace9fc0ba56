// gemm_mx_tile.hpp — tiled fused product of two MXFP4 operands on gfx950:
//   C[M,N] = act(A . B^T + bias (+ R)), both operands as rows of k (mx_args.hpp)
//
// Workgroup: WM x WN waves (m x n) of SJ x SI accumulator blocks of 32x32
// each: an output tile of 32 SJ WM (m) x 32 SI WN (n).  A k-step is two groups of
// 128 values, 128 bytes of codes and 8 scale bytes a row: a whole cache line
// per row.  (With one group a step, 64 bytes a row, a CU reads at half the rate:
// 68 against 133 GB/s measured from L2.)
//
// Codes reach LDS without passing through registers, 16 bytes a lane, two
// stages deep; chunk c of row r lies at slot c ^ (r & 7), which spreads the same
// chunk of eight neighbouring rows over all slots.  Rows 8 apart share a slot, and
// the counters show 4.5 conflict cycles per LDS instruction: reads of such
// fragments and nothing else reach 285 B/ns a CU, 318 with slot c ^ ((r >> 1) & 7),
// 321 in a row.  The four
// v_mfma_scale_f32_32x32x64 of a step take chunk ks of the step's first group in
// the lower half of a wave and chunk ks of its second group in the upper half:
// each lane then needs one scale word per row and step, whose byte ks the
// instruction's operand selector picks.  Scales travel 16 bytes a row for two
// steps at once, through registers: fetched with each step they would touch
// one cache line per row, as many as the codes do.
//
// Epilogue: each lane adds the bias, applies the activation to its own sums and
// puts the rounded values into LDS (16-byte chunk c of row r at slot c ^ r, within
// the row), from where whole rows are stored, 16 bytes a lane.  A residual comes in
// the same way: whole rows into LDS, then each value to the lane that holds its
// sum.  16-bit outputs take one pass, 32-bit ones a pass for each wm.  Both have
// the non-temporal policy: 32768x4096x1024 with a residual 150 us, 172 without.
//
// Measured, 256x256 tiles, bf16 outputs: 4096^3 with GELU 47.2 us (2.9 PFLOP/s),
// 40 without an activation; a step costs a round of tiles 1.9 us, 4.5 PFLOP/s,
// where these instructions alone reach 5.6 to 6.1 on random operands (8.3 to 8.6 on
// zeros: it is power that bounds them).  The rest of a round is its epilogue: 3.3 us for
// the sums' way through LDS, 3 to 5 for 33 MB of outputs, 6 for GELU's
// instructions.  32768x4096x1024 takes 125 us, eight rounds.  Workgroups that
// walk over tiles, the next one's first loads ahead of the stores, took as long
// (130 us), since a later load returns after all earlier stores; products of one
// round took 1 us longer.
#pragma once

#include "epilogue.hpp"
#include "gemm_mx.hpp"

namespace biasact {

namespace mxt {
template <int WM, int WN, int SJ, int SI>
struct Tile {
  static constexpr int THREADS = 64 * WM * WN, BM = 32 * SJ * WM, BN = 32 * SI * WN;
  static constexpr int A_STAGE = BM * 128, B_STAGE = BN * 128, S_BUF = (BM + BN) * 16;
  static constexpr int A_OFF = 0, B_OFF = 2 * A_STAGE, S_OFF = B_OFF + 2 * B_STAGE;
  static constexpr int BIAS_OFF = S_OFF + 2 * S_BUF, LDS_BYTES = BIAS_OFF + BN * 4;
  static_assert(BN <= THREADS, "bias");
  static constexpr int A_LOADS = BM * 128 / 16 / THREADS, B_LOADS = BN * 128 / 16 / THREADS;   // per wave and step
  static constexpr int S_LOADS = (BM + BN) / THREADS;                                          // scale rows per thread
  static_assert((BM + BN) % THREADS == 0, "scale rows");
  static_assert(BM * BN * 2 <= BIAS_OFF && 32 * SJ * BN * 4 <= BIAS_OFF, "epilogue staging");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

constexpr int WAIT_LGKM0 = 0xC07F;
constexpr int wait_vm(int n) { return 0x0F70 | (n & 0xF) | ((n >> 4) << 14); }

// 16 bytes per lane from off of the buffer to lds + 16 * lane
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
}

// 16 bytes that this kernel touches once (cache policy "non-temporal")
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
  if constexpr (DTO == DT_F16) {
    asm("" : "+v"(lo), "+v"(hi));                      // as in narrow: fp32 first
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), f16x2));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), mx::bf16x2));
  }
}

// acc += b . a^T over 64 k, scale byte KS of each word
template <int KS>
__device__ __forceinline__ f32x16 mfma32(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa) {
  const i32x8 x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const i32x8 y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, KS, (int)sb, KS, (int)sa);
}
}  // namespace mxt

template <int DTO, int WM, int WN, int SJ, int SI>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx_tile_kernel(MxGemmArgs a) {
  using T = mxt::Tile<WM, WN, SJ, SI>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS_BYTES];

  uint32_t tm, tn;
  map_tile(blockIdx.x, gridDim.x, a.tiles_m, a.tiles_n, tm, tn);
  const uint32_t m0 = tm * T::BM, n0 = tn * T::BN;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const int half = lane >> 5, lrow = lane & 31;
  const int G = (int)a.G;                     // >= 1

  // sums of n = 32 si + 8 (e / 4) + 4 half + e % 4, m = 32 sj + lrow of the wave's block
  f32x16 acc[SI][SJ];
#pragma unroll
  for (int si = 0; si < SI; ++si)
#pragma unroll
    for (int sj = 0; sj < SJ; ++sj)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[si][sj][r] = 0.0f;

  // ---- direct loads: 8 rows of 128 bytes each ---------------------------------------
  // Rows past the end read as zeros (or, where a huge offset wraps, as other
  // rows); their sums are not stored.  The main loop has no branches: loads for
  // which there is no step have a buffer of no bytes, i.e. fetch nothing.
  const uint32_t chunk = (lane & 7) ^ (lane >> 3);     // that goes to slot lane % 8 of row lane / 8
  const uint32_t a_off = (m0 + T::A_LOADS * 8 * w + (lane >> 3)) * a.G * 64u + chunk * 16u;
  const uint32_t b_off = (n0 + T::B_LOADS * 8 * w + (lane >> 3)) * a.G * 64u + chunk * 16u;
  constexpr int LOADS = T::A_LOADS + T::B_LOADS;
  // loads [from, to) of this wave's share of step s, into stage st
  auto issue = [&](int s, int st, int from, int to) {
    const bool more = 2 * s < G;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A, more ? a.a_bytes : 0u);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B, more ? a.b_bytes : 0u);
    // with an odd G the last step's second group reads as zero
    const bool cut = 2 * s + 1 >= G && chunk >= 4u;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if (i < from || i >= to) continue;
      if (i < T::A_LOADS)
        mxt::load_to_lds(ra, smem + T::A_OFF + st * T::A_STAGE + (T::A_LOADS * w + i) * 1024,
                         cut ? kOOB : a_off + (8u * i * a.G * 64u + s * 128u));
      else
        mxt::load_to_lds(rb, smem + T::B_OFF + st * T::B_STAGE + (T::B_LOADS * w + i - T::A_LOADS) * 1024,
                         cut ? kOOB : b_off + (8u * (i - T::A_LOADS) * a.G * 64u + s * 128u));
    }
  };

  // ---- scales: thread t brings rows t (and t + THREADS) of A's rows followed by B's ---
  // Words 4 S .. 4 S + 3 of the row, zero from G on.  first: S == 0 and any G, a
  // load never goes past the row's own words.  Else G > 4, and a load that would
  // brings the row's last four, shifted down by put_scales.
  auto load_scales = [&](int S, bool first, u32x4 (&v)[T::S_LOADS]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < T::S_LOADS; ++i) {
      const int row0 = i * T::THREADS + 64 * w;        // uniform; BM and BN are multiples of 64
      const bool of_a = row0 < T::BM, any = first || 4 * S < G;
      const __amdgpu_buffer_rsrc_t rs =
          of_a ? make_rsrc(a.As, any ? a.as_bytes : 0u) : make_rsrc(a.Bs, any ? a.bs_bytes : 0u);
      const uint32_t row = of_a ? m0 + row0 + lane : n0 + (row0 - T::BM) + lane;
      if (!first) {
        v[i] = ld_b128(rs, (row * a.G + min(4 * S, G - 4)) * 4u);
      } else if (G >= 4) {
        v[i] = ld_b128(rs, row * a.G * 4u);
      } else {
        v[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < G) v[i][e] = ld_b32(rs, (row * a.G + e) * 4u);
      }
    }
  };
  auto put_scales = [&](int S, const u32x4 (&v)[T::S_LOADS]) __attribute__((always_inline)) {
    const int d = S == 0 ? 0 : 4 * S - min(4 * S, G - 4);
    const bool one = d & 1, two = d & 2;               // uniform
#pragma unroll
    for (int i = 0; i < T::S_LOADS; ++i) {
      u32x4 o = v[i];
      o = one ? u32x4{o.y, o.z, o.w, 0u} : o;
      o = two ? u32x4{o.z, o.w, 0u, 0u} : o;
      *reinterpret_cast<u32x4*>(smem + T::S_OFF + (S & 1) * T::S_BUF + (i * T::THREADS + 64 * w + lane) * 16) = o;
    }
  };

  // ---- LDS fragment addresses: row, chunk 4 half + ks ------------------------------
  const uint32_t fr = lrow * 128 + (((4 * half) ^ (lrow & 7)) * 16);
  const uint32_t a_rd = T::A_OFF + wm * 32 * SJ * 128 + fr, b_rd = T::B_OFF + wn * 32 * SI * 128 + fr;

  // ---- main loop ---------------------------------------------------------------------
  // Step s: quarters 0 .. 2 multiply while the next quarter's fragments are read.
  // Then the one barrier, after this wave's loads of step s + 1 have landed and
  // its reads of step s are done: from there on stage s + 1 may be read and
  // stage s overwritten.  The first fragments of s + 1 and half the loads of
  // s + 2 go out before quarter 3 multiplies, the other half before the next
  // quarter: four loads a wave are what the address unit takes in one quarter,
  // and more would hold up the reads behind them.  Scale words of the next two
  // steps are loaded in even steps and put in odd ones, before the barrier that
  // their readers pass.
  const int steps = (G + 1) >> 1;
  u32x4 snext[T::S_LOADS];
  // this tile's bias (zeros past N or without one): its bits now, fp32 into LDS later
  const __amdgpu_buffer_rsrc_t rbias = make_rsrc(a.bias, a.bias_dt >= 0 ? a.bias_bytes : 0u);
  const uint32_t bias_n = n0 + threadIdx.x;
  const bool bias_ok = threadIdx.x < T::BN && bias_n < a.N;
  uint32_t bias;
  if (a.bias_dt == DT_F32) bias = ld_b32(rbias, bias_ok ? bias_n * 4u : kOOB);
  else bias = ld_b16(rbias, bias_ok ? bias_n * 2u : kOOB);
  load_scales(0, true, snext);
  issue(0, 0, 0, LOADS);
  put_scales(0, snext);
  if (threadIdx.x < T::BN)
    *reinterpret_cast<float*>(smem + T::BIAS_OFF + threadIdx.x * 4) =
        a.bias_dt == DT_F16 ? widen<DT_F16>(bias) : a.bias_dt == DT_BF16 ? widen<DT_BF16>(bias) : widen<DT_F32>(bias);
  const uint32_t sc_rd = T::S_OFF + lrow * 16 + half * 4;
  u32x4 fa[2][SJ], fb[2][SI];                          // by parity of the quarter
  uint32_t wa[2][SJ], wb[2][SI];                       // scale words, by parity of the step
  auto read = [&](int ks, int odd) __attribute__((always_inline)) {
    uint32_t ar = a_rd, br = b_rd;
    if constexpr (SJ * SI > 4) asm volatile("" : "+v"(ar), "+v"(br));   // no registers for each chunk's address
#pragma unroll
    for (int si = 0; si < SI; ++si)
      fb[ks & 1][si] = *reinterpret_cast<const u32x4*>(smem + (br ^ (16u * ks)) + odd * T::B_STAGE + si * 4096);
#pragma unroll
    for (int sj = 0; sj < SJ; ++sj)
      fa[ks & 1][sj] = *reinterpret_cast<const u32x4*>(smem + (ar ^ (16u * ks)) + odd * T::A_STAGE + sj * 4096);
  };
  auto read_scales = [&](int s, int odd) __attribute__((always_inline)) {
    const uint8_t* sp = smem + sc_rd + ((s >> 1) & 1) * T::S_BUF + odd * 8;
#pragma unroll
    for (int si = 0; si < SI; ++si)
      wb[odd][si] = *reinterpret_cast<const uint32_t*>(sp + (T::BM + wn * 32 * SI + si * 32) * 16);
#pragma unroll
    for (int sj = 0; sj < SJ; ++sj)
      wa[odd][sj] = *reinterpret_cast<const uint32_t*>(sp + (wm * 32 * SJ + sj * 32) * 16);
  };
  auto multiply = [&](auto ks_c, int odd) __attribute__((always_inline)) {
    constexpr int ks = decltype(ks_c)::value;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int si = 0; si < SI; ++si)
#pragma unroll
      for (int sj = 0; sj < SJ; ++sj)
        acc[si][sj] = mxt::mfma32<ks>(fb[ks & 1][si], fa[ks & 1][sj], acc[si][sj], wb[odd][si], wa[odd][sj]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto join = [&] {
    __builtin_amdgcn_s_waitcnt(mxt::wait_vm(0));
    __builtin_amdgcn_s_waitcnt(mxt::WAIT_LGKM0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int s, int odd) __attribute__((always_inline)) {
    read(1, odd);
    if (odd == 0) load_scales((s >> 1) + 1, false, snext);
    issue(s + 1, odd ^ 1, LOADS / 2, LOADS);
    multiply(std::integral_constant<int, 0>{}, odd);
    read(2, odd);
    multiply(std::integral_constant<int, 1>{}, odd);
    read(3, odd);
    if (odd == 1) put_scales((s >> 1) + 1, snext);
    multiply(std::integral_constant<int, 2>{}, odd);
    join();
    read(0, odd ^ 1);                                  // (past the last step: whatever is there, unused)
    read_scales(s + 1, odd ^ 1);
    issue(s + 2, odd, 0, LOADS / 2);
    multiply(std::integral_constant<int, 3>{}, odd);
  };
  join();
  read(0, 0);
  read_scales(0, 0);
  issue(1, 1, 0, LOADS / 2);
  for (int s = 0; s < steps; s += 2) {
    step(s, 0);
    if (s + 1 < steps) step(s + 1, 1);
  }
  // no direct load (of zeros) may still be writing LDS when the epilogue reuses it
  __builtin_amdgcn_s_waitcnt(mxt::wait_vm(0));

  // ---- epilogue -------------------------------------------------------------------
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.C, a.c_bytes);
  const __amdgpu_buffer_rsrc_t rr = make_rsrc(a.R, a.R ? a.c_bytes : 0u);
  constexpr int ES = Elem<DTO>::bytes, EPC = 16 / ES;  // bytes an output, outputs a chunk
  constexpr int CPR = T::BN / EPC;                     // chunks, and lanes, a row
  constexpr int PASSES = ES == 2 ? 1 : WM, ROWS = T::BM / PASSES;
  // whole 16-byte accesses: rows of whole chunks, aligned bases
  const bool vec = a.N % EPC == 0 && ((reinterpret_cast<uintptr_t>(a.C) | reinterpret_cast<uintptr_t>(a.R)) & 15u) == 0;
  // The thread's number, told to the compiler anew: addresses computed from it
  // here would otherwise be kept in registers through the main loop.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  auto slot = [](int r, int c) { return (uint32_t)(r * (T::BN * ES) + ((c ^ (r & (CPR - 1))) << 4)); };
  // f(LDS address, element offset in C, whether there is such an output), for
  // every chunk of the pass's rows, a row's chunks in neighbouring lanes
  constexpr int CHUNKS = ROWS * CPR / T::THREADS;
  auto by_chunk = [&](int pass, int from, int count, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < count; ++i) {
      const int r = (from + i) * (T::THREADS / CPR) + tid / CPR, c = tid % CPR;
      const uint32_t m = m0 + pass * ROWS + r, n = n0 + c * EPC;
      f(i, slot(r, c), m * a.N + n, m < a.M && n < a.N);
    }
  };
  // the same for every single output, a wave's 64 E of count rows at a time
  constexpr int E = T::BN / 64;
  auto by_output = [&](int pass, int from, int count, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < count * E; ++i) {
      const int r = (from + i / E) * (WM * WN) + w, c = (tid & 63) + 64 * (i % E);
      const uint32_t m = m0 + pass * ROWS + r, n = n0 + c;
      f(i, slot(r, c / EPC) + (c % EPC) * ES, m * a.N + n, m < a.M && n < a.N);
    }
  };
#pragma unroll 1
  for (int pass = 0; pass < PASSES; ++pass) {
    asm volatile("" : "+v"(tid));
    const int row = tid & 31, four = 4 * ((tid >> 5) & 1);
    __syncthreads();                                   // the last k-step, or the previous pass, is read
    if (a.R) {
      // eight or more loads at a time: a write to LDS waits for all earlier loads
      if (vec) {
#pragma unroll 1
        for (int from = 0; from < CHUNKS; from += 8) {
          u32x4 v[8];
          by_chunk(pass, from, 8, [&](int i, uint32_t, uint32_t at, bool ok) { v[i] = mxt::load_once(rr, ok ? at * ES : kOOB); });
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
      with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act_c)::value;
        with_residual(a.R != nullptr, [&](auto res_c) __attribute__((always_inline)) {
#pragma unroll
          for (int si = 0; si < SI; ++si)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int n = (wn * SI + si) * 32 + 8 * g + four;
              const f32x4 bias = *reinterpret_cast<const f32x4*>(smem + T::BIAS_OFF + n * 4);
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
                    o[e] = mxt::narrow2<DTO>(mx::act<ACT, DTO>(z[2 * e], a.alpha), mx::act<ACT, DTO>(z[2 * e + 1], a.alpha));
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
          mxt::store_once(rc, ok ? at * ES : kOOB, *reinterpret_cast<const u32x4*>(smem + p));
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

template <int DTO, int WM, int WN, int SJ, int SI>
inline void launch_mx_tile(MxGemmArgs a, hipStream_t s) {
  using T = mxt::Tile<WM, WN, SJ, SI>;
  a.tiles_n = (a.N + T::BN - 1) / T::BN;
  a.tiles_m = (a.M + T::BM - 1) / T::BM;
  note_launch("gemm mxfp4 tile, %d m x %d n", T::BM, T::BN);
  launch_kernel(mx_tile_kernel<DTO, WM, WN, SJ, SI>, dim3(a.tiles_m * a.tiles_n), dim3(T::THREADS), s, a);
}

}  // namespace biasact
