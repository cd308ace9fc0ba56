// act_grad.hip — gradient of the bias-and-activation epilogue act(z), and the
// sums of column parts that gradients of broadcast vectors end with.
//   dz = dy act'(z),  dbias = sum over rows of dz (before it is rounded)
#include "launch_kernel.hpp"
#include "norm_args.hpp"
#include "norm_plan.hpp"
#include "row_io.hpp"

namespace biasact {
namespace {

// e^-x for x >= 0: the product with log2 e in two parts, so that the exponent's
// rounding does not show in the result; zero (as from 104 on) past 200.
__device__ __forceinline__ float exp_neg(float x) {
#pragma clang fp contract(off)
  x = x > 200.0f ? 200.0f : x;
  const float hi = x * -1.442695022f;                  // log2 e = 1.442695022 + 1.925963e-8
  const float lo = __builtin_fmaf(x, -1.925963033e-8f, __builtin_fmaf(x, -1.442695022f, -hi));
  const float r = exp2_f32(hi);
  return __builtin_fmaf(r, lo * 0.693147181f, r);
}

// dy GELU'(z) = dy (Phi(z) + z phi(z)).  For x = |z|, GELU'(-x) = phi(x) (M(x) - x)
// and GELU'(x) = 1 - GELU'(-x), M the ratio of the normal distribution's tail to
// its density, as t Q(t), t = 1 / (1 + a x) (fit_mills.py): one exponential for both
// terms, and nothing cancels but at the slope's root.  Q is the same for every type:
// the bias's sums are fp32 whatever the type of dZ, and a degree that is enough for 16-bit dZ
// (6: 4e-6 of M, 62 times 2^-24) leaves its error in them.  fp32 tensors take x^2 in two
// parts, so that the exponent's rounding does not show; a 16-bit z has an exact x^2,
// and what the exponent's own rounding leaves, 0.61 x^2 2^-24 of phi, is large only
// where phi counts for nothing in a sum (8192x16384 bf16 171 to 176 us with those steps,
// 162 to 164 without).  Below 2^-126 the result is formed at 2^64 times its size, so that
// it rounds once (see exp2_f32).
template <int DT>
__device__ __forceinline__ float gelu_grad(float dy, float z) {
#pragma clang fp contract(off)
  float x = __builtin_fabsf(z);
  x = x > 60.0f ? 60.0f : x;                           // (phi is zero from 15 on; infinity times it is not)
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(x, 0.32f, 1.0f));
  float q = -5.283590034e-02f;
  q = __builtin_fmaf(q, t, 2.391539961e-01f);
  q = __builtin_fmaf(q, t, -3.677475452e-01f);
  q = __builtin_fmaf(q, t, 1.637595743e-01f);
  q = __builtin_fmaf(q, t, -2.350982092e-02f);
  q = __builtin_fmaf(q, t, 1.470248997e-01f);
  q = __builtin_fmaf(q, t, 2.201547027e-01f);
  q = __builtin_fmaf(q, t, 2.873156667e-01f);
  q = __builtin_fmaf(q, t, 3.199985325e-01f);
  q = __builtin_fmaf(q, t, 3.199999928e-01f);
  const float xx = x * x, e = xx * -0.721347511f;      // log2 e / 2 = 0.721347511 + 9.6298e-9
  const bool tiny = e < -126.0f;
  float r = __builtin_amdgcn_exp2f(tiny ? e + 64.0f : e);
  if constexpr (DT == DT_F32) {
    const float lo = __builtin_fmaf(x, x, -xx);
    const float c = __builtin_fmaf(lo, -0.721347511f, __builtin_fmaf(xx, -9.6298e-9f, __builtin_fmaf(xx, -0.721347511f, -e)));
    r = __builtin_fmaf(r, c * 0.693147181f, r);
  }
  const float h = (0.398942280f * r) * __builtin_fmaf(t, q, -x);
  if (z < 0.0f) return tiny ? (dy * h) * 0x1p-64f : dy * h;
  return dy * (1.0f - (tiny ? h * 0x1p-64f : h));
}

// dy times the activation's slope at z.
template <int ACT, int DT>
__device__ __forceinline__ float act_grad(float dy, float z, float alpha) {
#pragma clang fp contract(off)
  if constexpr (ACT == ACT_RELU) {
    return z > 0.0f ? dy : 0.0f;
  } else if constexpr (ACT == ACT_LEAKY) {
    return z >= 0.0f ? dy : alpha * dy;
  } else if constexpr (ACT == ACT_TANH) {              // 1 - tanh^2 = 4 u / (1 + u)^2, u = e^-2|z|
    const float u = exp_neg(2.0f * __builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + u);
    return dy * (4.0f * u * r * r);
  } else if constexpr (ACT == ACT_SIGMOID) {           // s (1 - s) = u / (1 + u)^2, u = e^-|z|
    const float u = exp_neg(__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + u);
    return dy * (u * r * r);
  } else if constexpr (ACT == ACT_GELU) {
    return gelu_grad<DT>(dy, z);
  } else {
    return dy;
  }
}

// A lane holds eight columns, 2^lane_bits lanes share a row, and a workgroup
// takes 256 >> lane_bits rows at once, walking down its share of them.  Bound by
// memory: dY and Z are read once, dZ written once.  bf16, us with the sums' join, beside
// a large copy's time for as many bytes (4.92 TB/s): 8192x16384 GELU 162 (164), 32768x4096
// LeakyReLU 151 (164), 1021x1003 tanh fp32 7.7, two launches.
template <int DT>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  __shared__ float cols[256][9];
  const uint32_t width = 1u << a.lane_bits, t = threadIdx.x & (width - 1u), sub = threadIdx.x >> a.lane_bits;
  const uint32_t once = 256u >> a.lane_bits;
  const uint32_t i = (blockIdx.x * width + t) * 8u;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  if (i < a.N)
    with_act(a.act, [&](auto act_c) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act_c)::value;
      for (uint32_t row = blockIdx.y * once + sub; row < a.M; row += a.parts * once) {
        const size_t base = (size_t)row * a.N;
        const Row8<DT> ry = load_row8<DT>(a.dY, base, i, a.N);
        Row8<DT> rz = ry;
        if constexpr (ACT != ACT_NONE) rz = load_row8<DT>(a.Z, base, i, a.N);
        float dz[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dz[e] = act_grad<ACT, DT>(value<DT>(ry, e), value<DT>(rz, e), a.alpha);
          s[e] += dz[e];
        }
        if (a.dZ) store_row8<DT>(a.dZ, base, i, a.N, dz);
      }
    });
  if (!a.part) return;                                 // uniform
#pragma unroll
  for (int e = 0; e < 8; ++e) cols[threadIdx.x][e] = s[e];
  __syncthreads();
  // column c of the workgroup's: the sums of its `once` rows in order
  for (uint32_t c = threadIdx.x; c < width * 8u; c += 256u) {
    const uint32_t col = blockIdx.x * width * 8u + c;
    if (col >= a.N) continue;
    float v = cols[c >> 3][c & 7u];
    for (uint32_t j = 1; j < once; ++j) v += cols[(j << a.lane_bits) + (c >> 3)][c & 7u];
    a.part[(size_t)blockIdx.y * a.N + col] = v;
  }
}

// 64 columns a workgroup at a time; each of its 16 waves adds every 16th part, and
// the waves' sums are added in order.  A few MB at most, from L2: 2.3 to 5.3 us
// (512 parts of 2 x 4096 columns 4.4 to 5.3).
__global__ __launch_bounds__(1024) void join_columns_kernel(JoinArgs a) {
  __shared__ float sums[2][16][64];
  const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
  void* const out = a.out[blockIdx.y];
  if (!out) return;                                    // uniform
  int odd = 0;
  for (uint32_t col0 = blockIdx.x * 64u; col0 < a.n; col0 += gridDim.x * 64u, odd ^= 1) {
    const uint32_t col = col0 + lane;
    float v = 0.0f;
    if (col < a.n) {
      const float* p = a.part + (size_t)w * a.stride + (size_t)blockIdx.y * a.n + col;
#pragma unroll 8
      for (uint32_t i = w; i < a.parts; i += 16u, p += (size_t)16 * a.stride) v += *p;
    }
    sums[odd][w][lane] = v;
    __syncthreads();                                   // (the next round's sums lie elsewhere)
    if (w || col >= a.n) continue;
    v = sums[odd][0][lane];
#pragma unroll
    for (int j = 1; j < 16; ++j) v += sums[odd][j][lane];
    if (a.dt == DT_F32) static_cast<float*>(out)[col] = v;
    else static_cast<uint16_t*>(out)[col] = (uint16_t)(a.dt == DT_F16 ? narrow<DT_F16>(v) : narrow<DT_BF16>(v));
  }
}

}  // namespace

int launch_act_grad(int dt, const ActGradArgs& a, hipStream_t s) {
  note_launch("bias and activation gradient, %u lanes a row, %u parts", 1u << a.lane_bits, a.parts);
  const uint32_t cols = 8u << a.lane_bits;
  const dim3 grid((a.N + cols - 1) / cols, a.parts), block(256);
  switch (dt) {
    case DT_F32: launch_kernel(act_grad_kernel<DT_F32>, grid, block, s, a); return 0;
    case DT_F16: launch_kernel(act_grad_kernel<DT_F16>, grid, block, s, a); return 0;
    case DT_BF16: launch_kernel(act_grad_kernel<DT_BF16>, grid, block, s, a); return 0;
    default: return -1;
  }
}

void launch_join_columns(const JoinArgs& a, hipStream_t s) {
  const uint32_t blocks = (a.n + 63u) / 64u;
  launch_kernel(join_columns_kernel, dim3(blocks < 65536u ? blocks : 65536u, a.out[1] ? 2u : 1u), dim3(1024), s, a);
}

}  // namespace biasact
