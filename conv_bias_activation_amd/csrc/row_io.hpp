// row_io.hpp — eight consecutive values of a row of any alignment, and sums over
// the threads of a row.
#pragma once

#include "device_common.hpp"

namespace biasact {

// Eight consecutive values as they are stored (16 or 32 bytes).
template <int DT> struct Row8 { uint32_t w[2 * Elem<DT>::bytes]; };

// Values i .. i + 7 of the n from p on, zero from n on.  p need only be aligned
// for one value: the copy lets the compiler use the widest load that a global
// address of any alignment takes.
template <int DT>
__device__ __forceinline__ Row8<DT> load_row8(const void* p, size_t base, uint32_t i, uint32_t n) {
  constexpr int ES = Elem<DT>::bytes;
  const uint8_t* src = static_cast<const uint8_t*>(p) + (base + i) * ES;
  Row8<DT> v;
  if (i + 8u <= n) {
    __builtin_memcpy(&v, src, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < 2 * ES; ++e) v.w[e] = 0;
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if (i + e < n) {
        if constexpr (ES == 4) v.w[e] = reinterpret_cast<const uint32_t*>(src)[e];
        else v.w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(src)[e] << (16 * (e & 1));
      }
  }
  return v;
}

// The same of a row of n values from element `base` of a tensor on (r: the whole of it,
// less than 2 GiB).  Where no piece is cut by the row's end (uniform), lanes past it read
// zeros without a branch: a branch's two sides write the same registers, so that a load
// for the next row would be waited for at once (layer norm gradient of 32768x768 bf16
// 60 us with the branch, 42 without; of 32768x4096, where no lane lies past it, 153 both).
template <int DT>
__device__ __forceinline__ Row8<DT> load_row8(__amdgpu_buffer_rsrc_t r, const void* p, uint32_t base, uint32_t i, uint32_t n) {
  constexpr int ES = Elem<DT>::bytes;
  if (n & 7u) return load_row8<DT>(p, (size_t)base, i, n);
  const uint32_t off = i < n ? (base + i) * ES : kOOB;
  Row8<DT> v;
#pragma unroll
  for (int h = 0; h < ES / 2; ++h) {
    const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16u * h, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) v.w[4 * h + e] = q[e];
  }
  return v;
}

template <int DT>
__device__ __forceinline__ float value(const Row8<DT>& v, int e) {
  if constexpr (DT == DT_F32) return __uint_as_float(v.w[e]);
  else return widen<DT>((v.w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
}

template <int DT>
__device__ __forceinline__ void store_row8(void* p, size_t base, uint32_t i, uint32_t n, const float (&y)[8]) {
  constexpr int ES = Elem<DT>::bytes;
  uint8_t* dst = static_cast<uint8_t*>(p) + (base + i) * ES;
  Row8<DT> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (ES == 4) v.w[e] = narrow<DT>(y[e]);
    else if (e & 1) v.w[e >> 1] |= narrow<DT>(y[e]) << 16;
    else v.w[e >> 1] = narrow<DT>(y[e]);
  }
  if (i + 8u <= n) {
    __builtin_memcpy(dst, &v, sizeof(v));
  } else {
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if (i + e < n) {
        if constexpr (ES == 4) reinterpret_cast<uint32_t*>(dst)[e] = v.w[e];
        else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(v.w[e >> 1] >> (16 * (e & 1)));
      }
  }
}

// Eight values of a vector that is fp32, fp16 or bf16 at run time (uniform), or
// `none` everywhere without one.
__device__ __forceinline__ void load_vec8(const void* p, int dt, uint32_t i, uint32_t n, float none, float (&o)[8]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = none;
  } else if (dt == DT_F32) {
    const Row8<DT_F32> v = load_row8<DT_F32>(p, 0, i, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = value<DT_F32>(v, e);
  } else if (dt == DT_F16) {
    const Row8<DT_F16> v = load_row8<DT_F16>(p, 0, i, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = value<DT_F16>(v, e);
  } else {
    const Row8<DT_BF16> v = load_row8<DT_BF16>(p, 0, i, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = value<DT_BF16>(v, e);
  }
}

// Sum over 16 neighbouring lanes, in each of them.
__device__ __forceinline__ float sum16(float x) {
  auto ror = [](float v, auto c) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), decltype(c)::value, 0xf, 0xf, true));
  };
  x += ror(x, std::integral_constant<int, 0x128>{});   // rotate 16 lanes by 8,
  x += ror(x, std::integral_constant<int, 0x124>{});   // 4,
  x += ror(x, std::integral_constant<int, 0x122>{});   // 2
  x += ror(x, std::integral_constant<int, 0x121>{});   // and 1
  return x;
}

// Sum over the T threads of a row (16, or whole waves), in each of them.  LDS of
// T / 64 floats a value is the caller's, its earlier readers done.
template <int T>
__device__ __forceinline__ void row_sum2(float& x, float& y, float* lds) {
  x = sum16(x);
  y = sum16(y);
  if constexpr (T >= 64) {
    x += __shfl_xor(x, 16);
    y += __shfl_xor(y, 16);
    x += __shfl_xor(x, 32);
    y += __shfl_xor(y, 32);
  }
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      lds[w] = x;
      lds[W + w] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      x += lds[i];
      y += lds[W + i];
    }
  }
}

}  // namespace biasact
