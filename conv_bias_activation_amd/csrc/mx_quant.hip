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
// lane 0 of the sixteen writes the group's four scale bytes as one word.  Bound
// by the bytes: 32768x4096 bf16 (340 MB) in 73.5 us, 4.6 TB/s where a copy of
// 2 GiB reaches 4.9; 4096x4096 in 8.0 us; one row of 4096 in 1.5 us, a launch.
// Read back, with the codes still in the caches, 56 and 1.5 us.
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
// A workgroup takes two groups of 128 k of 64 CPL columns, wave w their block w:
// a lane holds the block of its CPL columns, and consecutive lanes read
// consecutive values of each row of X.  CPL = 2 for 16-bit types, four bytes a
// load (an even number of columns, X aligned for them), else 1.  Codes and
// scales leave through LDS (block b of column c at slot b ^ (c / 2 % 8), which
// spreads a wave's writes over the banks), so that eight lanes store a
// column's whole cache line of codes; from the registers each store would touch
// 64 lines.  Bound by the bytes: 4096x4096 fp16 (42 MB, 8.7 us at 4.9 TB/s) in
// 9.4 us, 13.8 without these two; read back in 10.2.  With one column a lane, in
// graph replay: 4096x4096 fp32 12.8 us (15.7 for the bytes from HBM) and
// 16384x8192 fp32 125 (125), but a 16-bit X of odd width reads two bytes a lane:
// 4095x4096 fp16 12.8 us where 4096x4096 takes 8.0, 16383x8192 bf16 87 for 76.
template <int DT, int CPL>
__global__ __launch_bounds__(512) void mx_quantize_cols_kernel(MxQuantArgs a) {
  static_assert(CPL == 1 || Elem<DT>::bytes == 2, "two columns of a 16-bit type");
  constexpr uint32_t COLS = 64 * CPL;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[COLS * 136];
  const uint32_t lane = threadIdx.x & 63u, blk = threadIdx.x >> 6;
  const uint32_t d = fdiv(blockIdx.x, a.div_tiles), n0 = (blockIdx.x - d * a.div_tiles.div) * COLS;
  const uint32_t n = n0 + CPL * lane, k0 = d * 256u + blk * 32u;
  const bool in = n < a.rows;
  Raw8<DT> v[CPL][4];
#pragma unroll
  for (int c = 0; c < CPL; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 2 * Elem<DT>::bytes; ++i) v[c][q].w[i] = 0;
  uint32_t x[32];
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) {
    const size_t at = (size_t)(k0 + j) * a.rows + n;
    const bool ok = in && k0 + j < a.K;
    if constexpr (Elem<DT>::bytes == 4) x[j] = ok ? static_cast<const uint32_t*>(a.X)[at] : 0u;
    else if constexpr (CPL == 2) x[j] = ok ? static_cast<const uint32_t*>(a.X)[at >> 1] : 0u;
    else x[j] = ok ? static_cast<const uint16_t*>(a.X)[at] : 0u;
  }
#pragma unroll
  for (uint32_t j = 0; j < 32; ++j) {
    if constexpr (Elem<DT>::bytes == 4) {
      v[0][j >> 3].w[j & 7] = x[j];
    } else {
      v[0][j >> 3].w[(j & 7) >> 1] |= (x[j] & 0xffffu) << (16 * (j & 1));
      if constexpr (CPL == 2) v[1][j >> 3].w[(j & 7) >> 1] |= (x[j] >> 16) << (16 * (j & 1));
    }
  }
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) m = max(m, max_abs_bits<DT>(v[c][q]));
    const uint32_t byte = scale_byte<DT>(m), col = CPL * lane + c;
    const u32x4 o = {encode8<DT>(v[c][0], byte), encode8<DT>(v[c][1], byte), encode8<DT>(v[c][2], byte),
                     encode8<DT>(v[c][3], byte)};
    *reinterpret_cast<u32x4*>(lds + col * 128u + ((blk ^ ((col >> 1) & 7u)) << 4)) = o;
    lds[COLS * 128u + col * 8u + blk] = (uint8_t)byte;
  }
  __syncthreads();
#pragma unroll
  for (uint32_t c = threadIdx.x >> 3; c < COLS; c += 64) {
    const uint32_t b = threadIdx.x & 7u;
    if (n0 + c < a.rows && 2 * d + (b >> 2) < a.G)
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.codes) + ((size_t)(n0 + c) * a.G + 2 * d) * 64u + b * 16u) =
          *reinterpret_cast<const u32x4*>(lds + c * 128u + ((b ^ ((c >> 1) & 7u)) << 4));
  }
  const uint32_t c = threadIdx.x >> 1, half = threadIdx.x & 1u;
  if (c < COLS && n0 + c < a.rows && 2 * d + half < a.G)
    static_cast<uint32_t*>(a.scales)[(size_t)(n0 + c) * a.G + 2 * d + half] =
        *reinterpret_cast<const uint32_t*>(lds + COLS * 128u + c * 8u + half * 4u);
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
  } else if (back) {
    launch_kernel(mx_dequantize_cols_kernel<DT>, dim3(a.div_tiles.div * a.G), dim3(256), s, a);
  } else {
    constexpr int CPL = Elem<DT>::bytes == 2 ? 2 : 1;
    const bool pairs = CPL == 2 && a.rows % 2 == 0 && (reinterpret_cast<uintptr_t>(a.X) & 3u) == 0;
    MxQuantArgs b = a;
    if (pairs) b.div_tiles = make_fastdiv((a.rows + 127u) / 128u);
    const dim3 grid(b.div_tiles.div * ((a.G + 1u) / 2u));
    if (pairs) launch_kernel(mx_quantize_cols_kernel<DT, CPL>, grid, dim3(512), s, b);
    else launch_kernel(mx_quantize_cols_kernel<DT, 1>, grid, dim3(512), s, b);
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
