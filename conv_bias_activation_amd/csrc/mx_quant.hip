// mx_quant.hip — quantisation to MXFP4 and reading it back.
//
// Per block of 32 values: e = floor(log2 max|x|) - 2 (the exponent of the
// largest value, less that of the largest code, 6 = 1.5 * 2^2), clamped to
// [-127, 127]; the scale byte is e + 127, and a code is x / 2^e rounded to the
// nearest of the eight magnitudes, ties to the even code, anything above 6 to
// 6.  Both steps are exact up to that one rounding: the division only changes
// the exponent.  A block of zeros has scale byte 0, a block that holds an
// infinity or a NaN has scale byte 255 (NaN) and codes 0.
#include "launch_kernel.hpp"
#include "mx_args.hpp"
#include "mx_launch.hpp"

namespace biasact {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight consecutive values of one row as they are stored (16 or 32 bytes).
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

// Largest |x| of the eight as the bits of a non-negative value: magnitudes of
// one format order as integers, with infinity and NaN above every number.
template <int DT>
__device__ __forceinline__ uint32_t max_abs_bits(const Raw8<DT>& v) {
  uint32_t m = 0;
  if constexpr (Elem<DT>::bytes == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7fffffffu);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(v.w[i] & 0x7fffu, (v.w[i] >> 16) & 0x7fffu));
  }
  return m;
}

// Scale byte of a block whose largest magnitude has these bits.
template <int DT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if constexpr (DT == DT_F16) {
    if (m >= 0x7c00u) return 255u;
    m = __float_as_uint(widen<DT_F16>(m));      // exact: subnormals become normal fp32 values
  } else if constexpr (DT == DT_BF16) {
    m <<= 16;
  }
  const uint32_t e = m >> 23;                    // fp32 exponent field: floor(log2) + 127, or 0 below 2^-126
  if (e == 255u) return 255u;
  return e > 2u ? e - 2u : 0u;
}

// The eight codes, value 0 in the low four bits; the conversion divides by the
// power of two that the scale operand's exponent field holds.
template <int DT>
__device__ __forceinline__ uint32_t encode8(const Raw8<DT>& v, uint32_t byte) {
  if (byte == 255u) return 0u;
  const float s = __uint_as_float(byte << 23);
  uint32_t c = 0;
  if constexpr (DT == DT_F32) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[0]), __uint_as_float(v.w[1]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[2]), __uint_as_float(v.w[3]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[4]), __uint_as_float(v.w[5]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.w[6]), __uint_as_float(v.w[7]), s, 3);
  } else if constexpr (DT == DT_F16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v.w[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v.w[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v.w[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, v.w[3]), s, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v.w[3]), s, 3);
  }
  return c;
}

// Two values (byte SEL of the codes) in the output type's bits.
template <int DT, int SEL>
__device__ __forceinline__ void decode2(uint32_t codes, float s, Raw8<DT>& v) {
  if constexpr (DT == DT_F32) {
    const f32x2 x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, SEL);
    v.w[2 * SEL] = __float_as_uint(x[0]);
    v.w[2 * SEL + 1] = __float_as_uint(x[1]);
  } else if constexpr (DT == DT_F16) {
    v.w[SEL] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, SEL));
  } else {
    v.w[SEL] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
  }
}

template <int DT>
__device__ __forceinline__ Raw8<DT> decode8(uint32_t codes, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);     // exponent field 0 reads as 2^-127, 255 as NaN
  Raw8<DT> v;
  decode2<DT, 0>(codes, s, v);
  decode2<DT, 1>(codes, s, v);
  decode2<DT, 2>(codes, s, v);
  decode2<DT, 3>(codes, s, v);
  return v;
}

// ---- blocks along the rows of X[rows, K] ------------------------------------
// One lane per 8 values: four lanes make a block, sixteen a group of 128, and
// lane 0 of the sixteen writes the group's four scale bytes as one word.
template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(MxQuantArgs a) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= a.total) return;                        // total is a multiple of 16: whole groups leave
  const uint32_t row = fdiv(t, a.div_row);
  const uint32_t c = t - row * a.div_row.div;
  const uint32_t k0 = c * 8u;
  const uint8_t* src = static_cast<const uint8_t*>(a.X) + (size_t)row * a.K * Elem<DT>::bytes;
  Raw8<DT> v;
  if (k0 + 8u <= a.K) v = load8<DT>(src + (size_t)k0 * Elem<DT>::bytes);
  else v = load8_ragged<DT>(src, k0, a.K);
  uint32_t m = max_abs_bits<DT>(v);
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));   // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));   // lane ^ 2
  const uint32_t byte = scale_byte<DT>(m);
  static_cast<uint32_t*>(a.codes)[t] = encode8<DT>(v, byte);
  uint32_t s = byte << (8u * ((threadIdx.x >> 2) & 3u));
  s |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s, 0x124, 0xf, 0xf, true);         // rotate 16 lanes by 4
  s |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s, 0x128, 0xf, 0xf, true);         // and by 8
  if ((threadIdx.x & 15u) == 0) static_cast<uint32_t*>(a.scales)[t >> 4] = s;
}

template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_rows_kernel(MxQuantArgs a) {
  const uint32_t t = blockIdx.x * 256u + threadIdx.x;
  if (t >= a.total) return;
  const uint32_t row = fdiv(t, a.div_row);
  const uint32_t k0 = (t - row * a.div_row.div) * 8u;
  if (k0 >= a.K) return;
  const Raw8<DT> v = decode8<DT>(static_cast<const uint32_t*>(a.codes)[t], static_cast<const uint8_t*>(a.scales)[t >> 2]);
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

// ---- blocks down the columns of X[K, rows] ----------------------------------
// A lane holds one column's block of 32 k: consecutive lanes read consecutive
// values of each row of X.  Wave w of the workgroup takes block w of a group
// of 128, so the four waves fill a column's 64 bytes of codes.
template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_cols_kernel(MxQuantArgs a) {
  const uint32_t lane = threadIdx.x & 63u, blk = threadIdx.x >> 6;
  const uint32_t g = fdiv(blockIdx.x, a.div_tiles), n = (blockIdx.x - g * a.div_tiles.div) * 64u + lane;
  const uint32_t k0 = g * 128u + blk * 32u;
  if (n >= a.rows) return;
  Raw8<DT> v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 2 * Elem<DT>::bytes; ++i) v[q].w[i] = 0;
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) {
    if (k0 + j < a.K) {
      const size_t at = (size_t)(k0 + j) * a.rows + n;
      if constexpr (Elem<DT>::bytes == 4) v[j >> 3].w[j & 7] = static_cast<const uint32_t*>(a.X)[at];
      else v[j >> 3].w[(j & 7) >> 1] |= (uint32_t) static_cast<const uint16_t*>(a.X)[at] << (16 * (j & 1));
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) m = max(m, max_abs_bits<DT>(v[q]));
  const uint32_t byte = scale_byte<DT>(m);
  u32x4 o;
  o.x = encode8<DT>(v[0], byte);
  o.y = encode8<DT>(v[1], byte);
  o.z = encode8<DT>(v[2], byte);
  o.w = encode8<DT>(v[3], byte);
  *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.codes) + ((size_t)n * a.G + g) * 64u + blk * 16u) = o;
  static_cast<uint8_t*>(a.scales)[((size_t)n * a.G + g) * 4u + blk] = (uint8_t)byte;
}

template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_cols_kernel(MxQuantArgs a) {
  const uint32_t lane = threadIdx.x & 63u, blk = threadIdx.x >> 6;
  const uint32_t g = fdiv(blockIdx.x, a.div_tiles), n = (blockIdx.x - g * a.div_tiles.div) * 64u + lane;
  const uint32_t k0 = g * 128u + blk * 32u;
  if (n >= a.rows || k0 >= a.K) return;
  const u32x4 c = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.codes) + ((size_t)n * a.G + g) * 64u + blk * 16u);
  const uint32_t byte = static_cast<const uint8_t*>(a.scales)[((size_t)n * a.G + g) * 4u + blk];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const Raw8<DT> v = decode8<DT>(c[q], byte);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t k = k0 + q * 8 + e;
      if (k < a.K) {
        const size_t at = (size_t)k * a.rows + n;
        if constexpr (Elem<DT>::bytes == 4) static_cast<uint32_t*>(const_cast<void*>(a.X))[at] = v.w[e];
        else static_cast<uint16_t*>(const_cast<void*>(a.X))[at] = (uint16_t)(v.w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <int DT>
void launch(const MxQuantArgs& a, bool rows, bool back, hipStream_t s) {
  if (rows) {
    const dim3 grid((a.total + 255u) / 256u);
    if (back) launch_kernel(mx_dequantize_rows_kernel<DT>, grid, dim3(256), s, a);
    else launch_kernel(mx_quantize_rows_kernel<DT>, grid, dim3(256), s, a);
  } else {
    const dim3 grid(a.div_tiles.div * a.G);
    if (back) launch_kernel(mx_dequantize_cols_kernel<DT>, grid, dim3(256), s, a);
    else launch_kernel(mx_quantize_cols_kernel<DT>, grid, dim3(256), s, a);
  }
}

}  // namespace

int launch_mx_quant(int dt, const MxQuantArgs& a, bool rows, bool back, hipStream_t s) {
  note_launch("mxfp4 %s, blocks along %s", back ? "dequantize" : "quantize", rows ? "rows" : "columns");
  switch (dt) {
    case DT_F32: launch<DT_F32>(a, rows, back, s); return 0;
    case DT_F16: launch<DT_F16>(a, rows, back, s); return 0;
    case DT_BF16: launch<DT_BF16>(a, rows, back, s); return 0;
    default: return -1;
  }
}

}  // namespace biasact
