// f8_quant.hip — quantisation to 8-bit floating point in blocks of 128 and
// reading it back.
//
// Per block: the scale is the smallest power of two that brings the block's
// largest finite magnitude within the format's range, top = 1.75 * 2^P (P = 8 for
// e4m3, 15 for e5m2), its exponent clamped to [-127, 127]; a code is x / scale
// rounded to nearest, ties to even.  The division only changes the exponent, so
// there is one rounding, and nothing saturates.  An infinity becomes NaN in e4m3
// and stays one in e5m2, NaN stays NaN; neither counts for its block's scale.  A
// block without another value than zero has scale byte 0.
//
// Every kernel here is bound by memory and reads and writes each value once.  Times
// below are of calls replayed from a graph, beside what a large copy (4.92 TB/s, read and
// written bytes) would take for the same bytes.
#include "f8_launch.hpp"
#include "launch_kernel.hpp"

namespace biasact {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Eight consecutive values as they are stored (16 or 32 bytes).
template <int DT> struct Raw8 { uint32_t w[2 * Elem<DT>::bytes]; };

// p need only be aligned for one value: the copy lets the compiler use the
// widest load that a global address of any alignment takes.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const uint8_t* p) {
  Raw8<DT> v;
  __builtin_memcpy(&v, p, sizeof(v));
  return v;
}

// The values k0 .. k0 + 7 of a row of K, zero from K on.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_ragged(const uint8_t* row, uint32_t k0, uint32_t K) {
  constexpr int ES = Elem<DT>::bytes;
  Raw8<DT> v;
#pragma unroll
  for (int i = 0; i < 2 * ES; ++i) v.w[i] = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k0 + e < K) {
      if constexpr (ES == 4) v.w[e] = *reinterpret_cast<const uint32_t*>(row + (size_t)(k0 + e) * 4);
      else v.w[e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + (size_t)(k0 + e) * 2) << (16 * (e & 1));
    }
  return v;
}

// Bits of infinity in the stored type: magnitudes of one format order as
// integers, with infinity and NaN above every number.
template <int DT>
constexpr uint32_t kInfBits = DT == DT_F32 ? 0x7f800000u : DT == DT_F16 ? 0x7c00u : 0x7f80u;

// The magnitude's bits of value e of the eight.
template <int DT>
__device__ __forceinline__ uint32_t mag_bits(const Raw8<DT>& v, int e) {
  if constexpr (Elem<DT>::bytes == 4) return v.w[e] & 0x7fffffffu;
  else return (v.w[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
}

template <int DT, int NR>
__device__ __forceinline__ uint32_t max_bits(const Raw8<DT> (&v)[NR]) {
  if constexpr (Elem<DT>::bytes == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, mag_bits<DT>(v[i], e));
    return m;
  } else {                                             // two at a time
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i].w[e] & 0x7fff7fffu));
    return max((uint32_t)m.x, (uint32_t)m.y);
  }
}

// The same over the finite values.
template <int DT, int NR>
__device__ __forceinline__ uint32_t max_finite_bits(const Raw8<DT> (&v)[NR]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = mag_bits<DT>(v[i], e);
      m = max(m, b < kInfBits<DT> ? b : 0u);
    }
  return m;
}

// Bits of the largest finite magnitude, and whether any lane of the wave holds a
// value that is not finite (rare: only then are the values looked at one by one).
template <int DT, int NR>
__device__ __forceinline__ uint32_t top_bits(const Raw8<DT> (&v)[NR], bool& odd) {
  uint32_t m = max_bits<DT>(v);
  odd = __any(m >= kInfBits<DT>);
  if (__builtin_expect(odd, 0)) m = max_finite_bits<DT>(v);
  return m;
}

// Scale byte of a block whose largest finite magnitude has these bits.
template <int DT, int F8>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if constexpr (DT == DT_F16) m = __float_as_uint(widen<DT_F16>(m));      // exact: subnormals become normal fp32 values
  else if constexpr (DT == DT_BF16) m <<= 16;
  constexpr uint32_t P = F8 == DT_E4M3 ? 8u : 15u;
  const uint32_t e = (m >> 23) + ((m & 0x7fffffu) > 0x600000u ? 1u : 0u);   // one more past 1.75 * 2^floor(log2 m)
  return e > P ? e - P : 0u;
}

template <int DT>
__device__ __forceinline__ float value(const Raw8<DT>& v, int e) {
  if constexpr (DT == DT_F32) return __uint_as_float(v.w[e]);
  else return widen<DT>((v.w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
}

// The eight codes, value 0 in the lowest byte.  The conversion divides by the
// power of two that the scale operand's exponent field holds.
template <int DT, int F8, int I>
__device__ __forceinline__ s16x2 encode2(s16x2 c, const Raw8<DT>& v, float s) {
  constexpr bool hi = I & 1;
  if constexpr (DT == DT_F32) {
    const float x = __uint_as_float(v.w[2 * I]), y = __uint_as_float(v.w[2 * I + 1]);
    if constexpr (F8 == DT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x, y, s, hi);
    else return __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, x, y, s, hi);
  } else if constexpr (DT == DT_F16) {
    const f16x2 x = __builtin_bit_cast(f16x2, v.w[I]);
    if constexpr (F8 == DT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, x, s, hi);
    else return __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(c, x, s, hi);
  } else {
    const bf16x2 x = __builtin_bit_cast(bf16x2, v.w[I]);
    if constexpr (F8 == DT_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, x, s, hi);
    else return __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(c, x, s, hi);
  }
}

template <int DT, int F8>
__device__ __forceinline__ u32x2 encode8(const Raw8<DT>& v, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  s16x2 lo = {0, 0}, hi = {0, 0};
  lo = encode2<DT, F8, 0>(lo, v, s);
  lo = encode2<DT, F8, 1>(lo, v, s);
  hi = encode2<DT, F8, 2>(hi, v, s);
  hi = encode2<DT, F8, 3>(hi, v, s);
  return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// Codes of the values among the eight that are not finite, in their places.
template <int DT, int F8>
__device__ __forceinline__ u32x2 patch_nonfinite(const Raw8<DT>& v, u32x2 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = mag_bits<DT>(v, e);
    if (b >= kInfBits<DT>) {
      const uint32_t sign = __float_as_uint(value<DT>(v, e)) >> 31;
      const uint32_t code = (F8 == DT_E5M2 && b == kInfBits<DT> ? 0x7cu : 0x7fu) | (sign << 7);
      c[e >> 2] = (c[e >> 2] & ~(0xffu << (8 * (e & 3)))) | (code << (8 * (e & 3)));
    }
  }
  return c;
}

// Two values (word I / 2 of the codes, half I % 2) in the output type's bits.
template <int DT, int F8, int I>
__device__ __forceinline__ void decode2(u32x2 codes, float s, Raw8<DT>& v) {
  const uint32_t c = codes[I >> 1];
  constexpr bool hi = I & 1;
  if constexpr (DT == DT_F32) {
    f32x2 x;
    if constexpr (F8 == DT_E4M3) x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, hi);
    else x = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(c, s, hi);
    v.w[2 * I] = __float_as_uint(x[0]);
    v.w[2 * I + 1] = __float_as_uint(x[1]);
  } else if constexpr (DT == DT_F16) {
    if constexpr (F8 == DT_E4M3) v.w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, s, hi));
    else v.w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(c, s, hi));
  } else {
    if constexpr (F8 == DT_E4M3) v.w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, hi));
    else v.w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c, s, hi));
  }
}

template <int DT, int F8>
__device__ __forceinline__ Raw8<DT> decode8(u32x2 codes, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);     // exponent field 0 reads as 2^-127, 255 as NaN
  Raw8<DT> v;
  decode2<DT, F8, 0>(codes, s, v);
  decode2<DT, F8, 1>(codes, s, v);
  decode2<DT, F8, 2>(codes, s, v);
  decode2<DT, F8, 3>(codes, s, v);
  return v;
}

// Largest of 16 neighbouring lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xf, 0xf, true));   // rotate 16 lanes by 8,
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xf, 0xf, true));   // 4,
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x122, 0xf, 0xf, true));   // 2
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x121, 0xf, 0xf, true));  // and 1
}

// ---- X[rows, K], a scale for each 128 values of a row -----------------------------
// One lane per 8 values, a wave per 512 of a row: sixteen lanes make a block, and
// lane 0 writes the four scale bytes as one word.  32768x4096 bf16 70 us (copy 83;
// what was written just before is still in the last-level cache), 4096x4096 fp32 13.4 (17),
// 8x4096 bf16 2.2, which is a launch.
template <int DT, int F8>
__global__ __launch_bounds__(256) void f8_quantize_rows_kernel(F8QuantArgs a) {
  const uint32_t wid = blockIdx.x * 4u + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wid >= a.rows * a.KW) return;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t row = fdiv(wid, a.div), word = wid - row * a.KW;
  const uint32_t k0 = word * 512u + lane * 8u;
  const uint8_t* src = static_cast<const uint8_t*>(a.X) + (size_t)row * a.K * Elem<DT>::bytes;
  Raw8<DT> v[1];
  if (k0 + 8u <= a.K) v[0] = load8<DT>(src + (size_t)k0 * Elem<DT>::bytes);
  else v[0] = load8_ragged<DT>(src, k0, a.K);
  bool odd;
  const uint32_t byte = scale_byte<DT, F8>(max16(top_bits<DT>(v, odd)));
  u32x2 c = encode8<DT, F8>(v[0], byte);
  if (__builtin_expect(odd, 0)) c = patch_nonfinite<DT, F8>(v[0], c);
  if (k0 < a.KB * 128u)
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.codes) + (size_t)row * a.KB * 128u + k0) = c;
  const uint32_t s = (uint32_t)__builtin_amdgcn_readlane((int)byte, 0) | (uint32_t)__builtin_amdgcn_readlane((int)byte, 16) << 8 |
                     (uint32_t)__builtin_amdgcn_readlane((int)byte, 32) << 16 | (uint32_t)__builtin_amdgcn_readlane((int)byte, 48) << 24;
  if (lane == 0) static_cast<uint32_t*>(a.scales)[wid] = s;
}

// ---- X[rows, K], a scale for each 128 x 128 ---------------------------------------
// A workgroup per block, sixteen lanes a row, eight rows a thread: the block stays in
// registers between its maximum and its codes.  4096x4096 fp16 8.4 us (copy 10.2).
template <int DT, int F8>
__global__ __launch_bounds__(256) void f8_quantize_blocks_kernel(F8QuantArgs a) {
  __shared__ uint32_t part[4];
  const uint32_t rb = fdiv(blockIdx.x, a.div), kb = blockIdx.x - rb * a.KB;
  const uint32_t k0 = kb * 128u + (threadIdx.x & 15u) * 8u, row0 = rb * 128u + (threadIdx.x >> 4);
  Raw8<DT> v[8];
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) {
    const uint32_t row = row0 + 16u * i;
    const uint8_t* src = static_cast<const uint8_t*>(a.X) + (size_t)row * a.K * Elem<DT>::bytes;
    if (row < a.rows && k0 + 8u <= a.K) v[i] = load8<DT>(src + (size_t)k0 * Elem<DT>::bytes);
    else v[i] = load8_ragged<DT>(src, k0, row < a.rows ? a.K : 0u);
  }
  bool odd;
  uint32_t m = max16(top_bits<DT>(v, odd));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((threadIdx.x & 63u) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const uint32_t byte = scale_byte<DT, F8>(m);
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) {
    const uint32_t row = row0 + 16u * i;
    u32x2 c = encode8<DT, F8>(v[i], byte);
    if (__builtin_expect(odd, 0)) c = patch_nonfinite<DT, F8>(v[i], c);
    if (row < a.rows) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.codes) + (size_t)row * a.KB * 128u + k0) = c;
  }
  // the last block also writes the word's rest
  const uint32_t end = kb + 1 == a.KB ? a.KW * 4u : kb + 1;
  if (threadIdx.x < end - kb) static_cast<uint8_t*>(a.scales)[(size_t)rb * a.KW * 4u + kb + threadIdx.x] = (uint8_t)(threadIdx.x ? 0u : byte);
}

// Two neighbouring values of a row as they are stored, one word or two.
template <int DT> struct Pair { uint32_t w[Elem<DT>::bytes / 2]; };
template <int DT>
__device__ __forceinline__ Pair<DT> load_pair(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  Pair<DT> v;
  if constexpr (Elem<DT>::bytes == 4) {
    const u32x2 x = ld_b64(r, off);
    v.w[0] = x.x, v.w[1] = x.y;
  } else {
    v.w[0] = ld_b32(r, off);
  }
  return v;
}

// ---- X[K, rows]: blocks down the columns ------------------------------------------
// A workgroup takes 128 k of 128 columns: wave w the k from 32 w on, a lane two
// columns, so that a wave reads whole lines of X.  The columns' largest values (or, with
// a scale for 128 x 128, the tile's) meet in LDS.  Codes leave through LDS too, a
// column's 16-byte chunk c at slot c ^ (column / 2 % 8), so that eight lanes store the
// 128 bytes of a column.  4096 columns of 32768 bf16 85 us (copy 83; the same with two
// blocks of k a workgroup), 4096x4096 fp16 in 128 x 128 9.1 (10.2), 1001 columns of
// 333 fp16 3.7 (4.5 with two blocks), 4095 columns of 4096 fp16, whose pairs lie
// across words every other row, 12.5.
template <int DT, int F8>
__global__ __launch_bounds__(256) void f8_quantize_cols_kernel(F8QuantArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[128 * 128];
  __shared__ uint32_t most[4][128];
  const uint32_t lane = threadIdx.x & 63u, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t kb = fdiv(blockIdx.x, a.div), n0 = (blockIdx.x - kb * a.div.div) * 128u;
  const uint32_t n = n0 + 2u * lane, k0 = kb * 128u + 32u * w;
  // A pair need only be aligned for one value (the GPU runs with unaligned access
  // on).  The lane whose first column is the row's last takes the pair before it and
  // moves it down; a row of one column has no pair.
  constexpr uint32_t ES = Elem<DT>::bytes;
  const uint32_t bytes = a.K * a.rows * ES;
  const bool last = n + 1 == a.rows && a.rows > 1;
  const uint32_t off = n < a.rows ? (k0 * a.rows + n - (last ? 1u : 0u)) * ES : kOOB;
  Pair<DT> x[32];
  if (a.rows > 1) {                                    // uniform
#pragma unroll
    for (uint32_t j = 0; j < 32; ++j)
      x[j] = load_pair<DT>(make_rsrc(a.X, k0 + j < a.K ? bytes : 0u), n < a.rows ? off + j * a.rows * ES : kOOB);
    if (a.rows & 1u) {
#pragma unroll
      for (uint32_t j = 0; j < 32; ++j) {
        if constexpr (ES == 4) {
          x[j].w[0] = last ? x[j].w[1] : x[j].w[0];
        } else {
          x[j].w[0] = last ? x[j].w[0] >> 16 : x[j].w[0];
        }
      }
    }
  } else {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a.X, bytes);
#pragma unroll
    for (uint32_t j = 0; j < 32; ++j) {
      const uint32_t at = lane == 0 && k0 + j < a.K ? (k0 + j) * ES : kOOB;
      if constexpr (ES == 4) x[j].w[0] = ld_b32(r, at), x[j].w[1] = 0;
      else x[j].w[0] = ld_b16(r, at);
    }
  }
  Raw8<DT> v[2][4];
#pragma unroll
  for (uint32_t j = 0; j < 32; j += 2) {
    if constexpr (Elem<DT>::bytes == 4) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        v[c][j >> 3].w[j & 7] = x[j].w[c];
        v[c][j >> 3].w[(j & 7) + 1] = x[j + 1].w[c];
      }
    } else {
      v[0][j >> 3].w[(j & 7) >> 1] = __builtin_amdgcn_perm(x[j + 1].w[0], x[j].w[0], 0x05040100u);
      v[1][j >> 3].w[(j & 7) >> 1] = __builtin_amdgcn_perm(x[j + 1].w[0], x[j].w[0], 0x07060302u);
    }
  }
  uint32_t m[2];
  bool odd[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) m[c] = top_bits<DT>(v[c], odd[c]);
  *reinterpret_cast<u32x2*>(&most[w][2 * lane]) = u32x2{m[0], m[1]};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2 o = *reinterpret_cast<const u32x2*>(&most[i][2 * lane]);
    m[0] = max(m[0], o.x);
    m[1] = max(m[1], o.y);
  }
  if (a.sh) {                                          // uniform
    uint32_t t = max16(max(m[0], m[1]));
    t = max(t, (uint32_t)__shfl_xor((int)t, 16));
    m[0] = m[1] = max(t, (uint32_t)__shfl_xor((int)t, 32));
  }
  uint32_t byte[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    byte[c] = scale_byte<DT, F8>(m[c]);
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      u32x2 lo = encode8<DT, F8>(v[c][2 * h], byte[c]), hi = encode8<DT, F8>(v[c][2 * h + 1], byte[c]);
      if (__builtin_expect(odd[c], 0)) {
        lo = patch_nonfinite<DT, F8>(v[c][2 * h], lo);
        hi = patch_nonfinite<DT, F8>(v[c][2 * h + 1], hi);
      }
      *reinterpret_cast<u32x4*>(lds + (2 * lane + c) * 128u + (((2 * w + h) ^ (lane & 7u)) << 4)) = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
  // scale bytes; the row's last block also writes its word's rest
  if (w == 0) {
    uint8_t* const s = static_cast<uint8_t*>(a.scales);
    const uint32_t end = kb + 1 == a.KB ? a.KW * 4u : kb + 1;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const bool in = a.sh ? lane == 0 && c == 0 : n + c < a.rows;
      uint8_t* const at = s + (size_t)(a.sh ? n0 >> 7 : n + c) * a.KW * 4u;
      if (in) {
        at[kb] = (uint8_t)byte[c];
        for (uint32_t e = kb + 1; e < end; ++e) at[e] = 0;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t c = 32u * i + (threadIdx.x >> 3), q = threadIdx.x & 7u;
    if (n0 + c < a.rows)
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.codes) + ((size_t)(n0 + c) * a.KB + kb) * 128u + q * 16u) =
          *reinterpret_cast<const u32x4*>(lds + c * 128u + ((q ^ ((c >> 1) & 7u)) << 4));
  }
}

// ---- reading back -------------------------------------------------------------------
// Along the rows: eight codes a lane.  32768x4096 bf16 63 to 68 us (copy 83).
template <int DT, int F8>
__global__ __launch_bounds__(256) void f8_dequantize_rows_kernel(F8QuantArgs a) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= a.rows * a.KB * 16u) return;
  const uint32_t row = fdiv(t, a.div), c = t - row * a.div.div, k0 = c * 8u;
  if (k0 >= a.K) return;
  const uint32_t byte = static_cast<const uint8_t*>(a.scales)[(size_t)(row >> a.sh) * a.KW * 4u + (c >> 4)];
  const Raw8<DT> v = decode8<DT, F8>(static_cast<const u32x2*>(a.codes)[t], byte);
  uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(a.X)) + ((size_t)row * a.K + k0) * Elem<DT>::bytes;
  if (k0 + 8u <= a.K) {
    __builtin_memcpy(dst, &v, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k0 + e < a.K) {
        if constexpr (Elem<DT>::bytes == 4) reinterpret_cast<uint32_t*>(dst)[e] = v.w[e];
        else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(v.w[e >> 1] >> (16 * (e & 1)));
      }
  }
}

// Down the columns: a lane reads 16 codes of each of two columns, twice, a wave
// writes whole lines of X: 4096 columns of 32768 bf16 104 us (copy 83), 4096x4096
// fp16 10.4 (10.2).  (A workgroup takes 256 k, which keeps the grid of a
// single long column within 2^32 threads.)
template <int DT, int F8>
__global__ __launch_bounds__(512) void f8_dequantize_cols_kernel(F8QuantArgs a) {
  const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
  const uint32_t d = fdiv(blockIdx.x, a.div), n = (blockIdx.x - d * a.div.div) * 128u + 2u * lane;
  const bool two = n + 1 < a.rows;
#pragma unroll
  for (uint32_t h = 0; h < 2; ++h) {
    const uint32_t k0 = d * 256u + h * 128u + 16u * w, kb = 2u * d + h;
    if (n >= a.rows || k0 >= a.K) return;
    Raw8<DT> v[2][2];
#pragma unroll
    for (uint32_t c = 0; c < 2; ++c) {
      const uint32_t col = min(n + c, a.rows - 1u);
      const u32x4 q = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.codes) + ((size_t)col * a.KB + kb) * 128u + 16u * w);
      const uint32_t byte = static_cast<const uint8_t*>(a.scales)[(size_t)(col >> a.sh) * a.KW * 4u + kb];
      v[c][0] = decode8<DT, F8>(u32x2{q.x, q.y}, byte);
      v[c][1] = decode8<DT, F8>(u32x2{q.z, q.w}, byte);
    }
#pragma unroll
    for (uint32_t j = 0; j < 16; ++j) {
      if (k0 + j >= a.K) break;
      uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(a.X)) + ((size_t)(k0 + j) * a.rows + n) * Elem<DT>::bytes;
      if constexpr (Elem<DT>::bytes == 4) {
        const u32x2 o = {v[0][j >> 3].w[j & 7], v[1][j >> 3].w[j & 7]};
        if (two) __builtin_memcpy(dst, &o, 8);
        else *reinterpret_cast<uint32_t*>(dst) = o.x;
      } else {
        const uint32_t sh = 16 * (j & 1), i = (j & 7) >> 1;
        const uint32_t o = ((v[0][j >> 3].w[i] >> sh) & 0xffffu) | ((v[1][j >> 3].w[i] >> sh) << 16);
        if (two) __builtin_memcpy(dst, &o, 4);
        else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)o;
      }
    }
  }
}

template <int DT, int F8>
void launch(F8QuantArgs a, bool along_rows, bool back, hipStream_t s) {
  const uint32_t col_tiles = (a.rows + 127u) / 128u;
  if (!along_rows) {
    a.div = make_fastdiv(col_tiles);
    if (back) launch_kernel(f8_dequantize_cols_kernel<DT, F8>, dim3(col_tiles * ((a.KB + 1u) / 2u)), dim3(512), s, a);
    else launch_kernel(f8_quantize_cols_kernel<DT, F8>, dim3(col_tiles * a.KB), dim3(256), s, a);
  } else if (back) {
    a.div = make_fastdiv(a.KB * 16u);
    launch_kernel(f8_dequantize_rows_kernel<DT, F8>, dim3((a.rows * a.KB * 16u + 255u) / 256u), dim3(256), s, a);
  } else if (a.sh) {
    a.div = make_fastdiv(a.KB);
    launch_kernel(f8_quantize_blocks_kernel<DT, F8>, dim3(col_tiles * a.KB), dim3(256), s, a);
  } else {
    a.div = make_fastdiv(a.KW);
    launch_kernel(f8_quantize_rows_kernel<DT, F8>, dim3((a.rows * a.KW + 3u) / 4u), dim3(256), s, a);
  }
}

template <int F8>
int launch_f8(int dt, const F8QuantArgs& a, bool along_rows, bool back, hipStream_t s) {
  switch (dt) {
    case DT_F32: launch<DT_F32, F8>(a, along_rows, back, s); return 0;
    case DT_F16: launch<DT_F16, F8>(a, along_rows, back, s); return 0;
    case DT_BF16: launch<DT_BF16, F8>(a, along_rows, back, s); return 0;
    default: return -1;
  }
}

}  // namespace

int launch_f8_quant(int dt, int f8, const F8QuantArgs& a, bool along_rows, bool back, hipStream_t s) {
  note_launch("fp8 %s, blocks of %d along %s", back ? "dequantize" : "quantize", a.sh ? 128 : 1, along_rows ? "rows" : "columns");
  if (f8 == DT_E4M3) return launch_f8<DT_E4M3>(dt, a, along_rows, back, s);
  return launch_f8<DT_E5M2>(dt, a, along_rows, back, s);
}

}  // namespace biasact
