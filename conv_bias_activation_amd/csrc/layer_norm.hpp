// layer_norm.hpp — layer norm over the rows of X[rows, N], and its gradient.
//   y = (x - mean) rstd gamma + beta,  rstd = 1 / sqrt(var + eps)
// Statistics are fp32: first a mean m, then sums of x - m and of its square
// over the values held in registers.  The first corrects m by what its own
// rounding left (d), so that an offset that is large beside the deviation costs no
// accuracy: mean = m + d, var = sum (x - m)^2 / N - d^2.
#pragma once

#include "launch_kernel.hpp"
#include "norm_args.hpp"
#include "norm_plan.hpp"
#include "row_io.hpp"

namespace biasact {

// (Rounding can leave a variance just below zero; NaN stays NaN.)
__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.0f / __builtin_sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// T threads a row (16 or 64: several rows a workgroup of 256), C chunks of eight
// values a thread: rows of up to 8 T C values.  A workgroup walks rows with gamma and
// beta in registers, the next row's values coming in while it works on this one.
// Bound by memory: each value is read and written once.  bf16, us, beside the time of a
// large copy of as many bytes (4.92 TB/s): 32768x4096 95 to 100 (109; a workgroup a row 128),
// 32768x1024 25 (27; 44), 32768x2048 45 to 53 (55), 8192x8192 47 (55), 8192x5120 43 (34),
// 1x4096 3.0, a launch.
template <int DTX, int DTY, int T, int C>
__global__ __launch_bounds__(T > 256 ? T : 256) void layer_norm_kernel(NormArgs a) {
  constexpr int WG = T > 256 ? T : 256, W = T > 64 ? T / 64 : 1;
  __shared__ float part[2][2 * W];
  const uint32_t t = threadIdx.x % T, step = gridDim.x * (WG / T);
  uint32_t row = blockIdx.x * (WG / T) + threadIdx.x / T;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X, a.rows * a.N * Elem<DTX>::bytes);
  Row8<DTX> next[C];
  auto fetch = [&](uint32_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) next[c] = load_row8<DTX>(rx, a.X, r * a.N, (c * T + t) * 8u, a.N);
  };
  if (row < a.rows) fetch(row);
  float g[C][8], b[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_vec8(a.gamma, a.dtw, (c * T + t) * 8u, a.N, 1.0f, g[c]);
    load_vec8(a.beta, a.dtw, (c * T + t) * 8u, a.N, 0.0f, b[c]);
  }
  for (; row < a.rows; row += step) {                  // (whole rows leave; with one row a workgroup it leaves as a whole)
    float x[C][8], s = 0.0f, none = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[c][e] = value<DTX>(next[c], e);
        s += x[c][e];
      }
    if (row + step < a.rows) fetch(row + step);
    row_sum2<T>(s, none, part[0]);
    const float n = (float)a.N, m = s / n;
    float d = 0.0f, q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[c][e] = (c * T + t) * 8u + e < a.N ? x[c][e] - m : 0.0f;
        d += x[c][e];
        q = __builtin_fmaf(x[c][e], x[c][e], q);
      }
    row_sum2<T>(d, q, part[1]);
    d /= n;
    const float rstd = rstd_of(q / n - d * d, a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = (c * T + t) * 8u;
      if (i >= a.N) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf((x[c][e] - d) * rstd, g[c][e], b[c][e]);
      store_row8<DTY>(a.Y, (size_t)row * a.N, i, a.N, y);
    }
    if (t == 0 && a.mean) {
      a.mean[row] = m + d;
      a.rstd[row] = rstd;
    }
  }
}

// Rows too long for registers: a workgroup a row, which it reads three times, the second
// and third time from L2 where few rows are under way.  us, beside the copy's time for the
// bytes read and written once: 4096x18432 bf16 85 (61), fp32 161 (123), 2048x32768 bf16 74
// (55), 512x131072 81 (55), 64x32768 8.6 (1.7).
template <int DTX, int DTY>
__global__ __launch_bounds__(1024) void layer_norm_long_kernel(NormArgs a) {
  __shared__ float part[2][32];
  const uint32_t row = blockIdx.x;
  const size_t base = (size_t)row * a.N;
  float s = 0.0f, none = 0.0f;
  for (uint32_t i = threadIdx.x * 8u; i < a.N; i += 8192u) {
    const Row8<DTX> v = load_row8<DTX>(a.X, base, i, a.N);
    float o = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o += value<DTX>(v, e);
    s += o;
  }
  row_sum2<1024>(s, none, part[0]);
  const float n = (float)a.N, m = s / n;
  float d = 0.0f, q = 0.0f;
  for (uint32_t i = threadIdx.x * 8u; i < a.N; i += 8192u) {
    const Row8<DTX> v = load_row8<DTX>(a.X, base, i, a.N);
    float od = 0.0f, oq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = i + e < a.N ? value<DTX>(v, e) - m : 0.0f;
      od += x;
      oq = __builtin_fmaf(x, x, oq);
    }
    d += od;
    q += oq;
  }
  row_sum2<1024>(d, q, part[1]);
  d /= n;
  const float rstd = rstd_of(q / n - d * d, a.eps);
  for (uint32_t i = threadIdx.x * 8u; i < a.N; i += 8192u) {
    const Row8<DTX> v = load_row8<DTX>(a.X, base, i, a.N);
    float g[8], b[8], y[8];
    load_vec8(a.gamma, a.dtw, i, a.N, 1.0f, g);
    load_vec8(a.beta, a.dtw, i, a.N, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf((value<DTX>(v, e) - m - d) * rstd, g[e], b[e]);
    store_row8<DTY>(a.Y, base, i, a.N, y);
  }
  if (threadIdx.x == 0 && a.mean) {
    a.mean[row] = m + d;
    a.rstd[row] = rstd;
  }
}

template <int DTX, int DTY, int T, int C>
inline void launch_norm(const NormArgs& a, hipStream_t s) {
  // Four times what the CUs hold at once; with four chunks a thread, whose weights take
  // longer to load, ten workgroups a CU (us: 8192x8192 bf16 47, with 8192 workgroups 56;
  // 32768x4096, two chunks, 106 and 100).
  constexpr uint32_t WG = T > 256 ? T : 256, ONCE = WG / T, MOST = C == 4 ? 2560u : 256u * 8192u / WG;
  const uint32_t groups = (a.rows + ONCE - 1) / ONCE;
  note_launch("layer norm, %d threads a row, %d values a thread", T, 8 * C);
  launch_kernel(layer_norm_kernel<DTX, DTY, T, C>, dim3(groups < MOST ? groups : MOST), dim3(WG), s, a);
}

template <int DTX, int DTY>
inline void launch_norm_to(const NormArgs& a, hipStream_t s) {
  if (a.N > kNormLong) {
    note_launch("layer norm, long rows");
    return launch_kernel(layer_norm_long_kernel<DTX, DTY>, dim3(a.rows), dim3(1024), s, a);
  }
  if (a.N <= 128) return launch_norm<DTX, DTY, 16, 1>(a, s);
  if (a.N <= 512) return launch_norm<DTX, DTY, 64, 1>(a, s);
  if (a.N <= 1024) return launch_norm<DTX, DTY, 64, 2>(a, s);
  // With few rows more threads a row hide its latency (us: 1x4096 3.0 with 512, 3.4
  // with 256; 2048x4096 9.9 and 9.3; 64x8192 4.1 with 512, 5.0 with 256, 8192x8192 50 and
  // 47; 32768x2048 49 with 256, 45 with one wave).
  const bool few = a.rows < 2048;
  if (a.N <= 2048) return few ? launch_norm<DTX, DTY, 256, 1>(a, s) : launch_norm<DTX, DTY, 64, 4>(a, s);
  if (a.N <= 4096) return few ? launch_norm<DTX, DTY, 512, 1>(a, s) : launch_norm<DTX, DTY, 256, 2>(a, s);
  if (a.N <= 8192) return few ? launch_norm<DTX, DTY, 512, 2>(a, s) : launch_norm<DTX, DTY, 256, 4>(a, s);
  launch_norm<DTX, DTY, 1024, 2>(a, s);
}

template <int DTX>
inline int launch_layer_norm(int dty, const NormArgs& a, hipStream_t s) {
  switch (dty) {
    case DT_F32: launch_norm_to<DTX, DT_F32>(a, s); return 0;
    case DT_F16: launch_norm_to<DTX, DT_F16>(a, s); return 0;
    case DT_BF16: launch_norm_to<DTX, DT_BF16>(a, s); return 0;
    default: return -1;
  }
}

// ---- gradient ---------------------------------------------------------------------
//   g = dy gamma, xh = (x - mean) rstd
//   dx = rstd (g - sum(g) / N - xh sum(g xh) / N)
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
// A workgroup walks rows parts apart, T threads a row, and keeps the column sums
// of what it has seen in registers: X and dY are read once, dX written once, which is
// what bounds it.  Its sums go to part[workgroup], which a second kernel adds up in a fixed
// order (atomics would change it).  Both kernels, us, beside the copy's time for as many
// bytes: 32768x4096 bf16 150 to 157 (164; 175 without the next row under way), fp32 285
// (328), 32768x1024 bf16 37 (41), 4096x16384 bf16 95 (82), 1001x1024 fp32 9.8, two launches.
template <int DTX, int DTY, int T, int C>
__global__ __launch_bounds__(T > 256 ? T : 256) void layer_norm_grad_kernel(NormGradArgs a) {
  constexpr int WG = T > 256 ? T : 256, G = WG / T, W = T > 64 ? T / 64 : 1;
  __shared__ float part[2][2 * W];
  __shared__ float cols[G > 1 ? G : 1][G > 1 ? T * C * 8 : 1];
  const uint32_t t = threadIdx.x % T, grp = threadIdx.x / T;
  float g[C][8], dg[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_vec8(a.gamma, a.dtw, (c * T + t) * 8u, a.N, 1.0f, g[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[c][e] = db[c][e] = 0.0f;
  }
  const float inv_n = 1.0f / (float)a.N;
  // the next row's values come in while this one is worked on (AHEAD), but where
  // 1024 threads leave no registers for them
  constexpr bool AHEAD = T < 1024;
  const __amdgpu_buffer_rsrc_t bx = make_rsrc(a.X, a.rows * a.N * Elem<DTX>::bytes), by = make_rsrc(a.dY, a.rows * a.N * Elem<DTY>::bytes);
  Row8<DTX> nx[C];
  Row8<DTY> ny[C];
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto fetch = [&](uint32_t row) __attribute__((always_inline)) {
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = (c * T + t) * 8u;
      nx[c] = AHEAD ? load_row8<DTX>(bx, a.X, row * a.N, i, a.N) : load_row8<DTX>(a.X, (size_t)row * a.N, i, a.N);
      ny[c] = AHEAD ? load_row8<DTY>(by, a.dY, row * a.N, i, a.N) : load_row8<DTY>(a.dY, (size_t)row * a.N, i, a.N);
    }
  };
  const uint32_t first = blockIdx.x * G + grp, step = a.parts * G;
  if (AHEAD && first < a.rows) fetch(first);
  int odd = 0;
  for (uint32_t row = first; row < a.rows; row += step, odd ^= 1) {
    const size_t base = (size_t)row * a.N;
    if (!AHEAD) fetch(row);
    const float mean = next_mean, rstd = next_rstd;
    Row8<DTX> rx[C];
    Row8<DTY> ry[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      rx[c] = nx[c];
      ry[c] = ny[c];
    }
    if (AHEAD && row + step < a.rows) fetch(row + step);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (value<DTX>(rx[c], e) - mean) * rstd, dy = value<DTY>(ry[c], e);
        const bool in = (c * T + t) * 8u + e < a.N;    // (past N: x and dy read as zero, xh does not)
        const float gy = dy * g[c][e];
        s1 += in ? gy : 0.0f;
        s2 = __builtin_fmaf(in ? gy : 0.0f, in ? xh : 0.0f, s2);
        dg[c][e] = __builtin_fmaf(dy, xh, dg[c][e]);
        db[c][e] += dy;
      }
    row_sum2<T>(s1, s2, part[odd]);
    s1 *= inv_n;
    s2 *= inv_n;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t i = (c * T + t) * 8u;
      if (i >= a.N) continue;
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (value<DTX>(rx[c], e) - mean) * rstd;
        dx[e] = rstd * (value<DTY>(ry[c], e) * g[c][e] - s1 - xh * s2);
      }
      store_row8<DTX>(a.dX, base, i, a.N, dx);
    }
  }
  if (!a.part) return;                                 // uniform
  float* const out = a.part + (size_t)blockIdx.x * 2u * a.N;
  // the groups' sums meet in LDS, in group order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (G > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) cols[grp][(c * T + t) * 8 + e] = which ? db[c][e] : dg[c][e];
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < a.N; i += WG) {
        float s = cols[0][i];
#pragma unroll
        for (int j = 1; j < G; ++j) s += cols[j][i];
        out[which * a.N + i] = s;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if ((c * T + t) * 8u < a.N) store_row8<DT_F32>(out, (size_t)which * a.N, (c * T + t) * 8u, a.N, which ? db[c] : dg[c]);
    }
  }
}

// Rows too long for registers: dX with a workgroup a row, which it reads twice; the
// column sums by a kernel of their own, which reads X and dY once more.  All three kernels,
// us, beside the copy's time for X, dY and dX once: 4096x18432 bf16 178 (92; 113 for dX, 64 and
// 5 for the sums), fp32 349 (184), 2048x32768 bf16 156 (82), 512x131072 201 (82), 64x32768 24 (2.6).
template <int DTX, int DTY>
__global__ __launch_bounds__(1024) void layer_norm_grad_long_kernel(NormGradArgs a) {
  __shared__ float part[32];
  const uint32_t row = blockIdx.x;
  const size_t base = (size_t)row * a.N;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (uint32_t i = threadIdx.x * 8u; i < a.N; i += 8192u) {
    const Row8<DTX> rx = load_row8<DTX>(a.X, base, i, a.N);
    const Row8<DTY> ry = load_row8<DTY>(a.dY, base, i, a.N);
    float g[8], o1 = 0.0f, o2 = 0.0f;
    load_vec8(a.gamma, a.dtw, i, a.N, 1.0f, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool in = i + e < a.N;
      const float gy = in ? value<DTY>(ry, e) * g[e] : 0.0f, xh = in ? (value<DTX>(rx, e) - mean) * rstd : 0.0f;
      o1 += gy;
      o2 = __builtin_fmaf(gy, xh, o2);
    }
    s1 += o1;
    s2 += o2;
  }
  row_sum2<1024>(s1, s2, part);
  const float inv_n = 1.0f / (float)a.N;
  s1 *= inv_n;
  s2 *= inv_n;
  for (uint32_t i = threadIdx.x * 8u; i < a.N; i += 8192u) {
    const Row8<DTX> rx = load_row8<DTX>(a.X, base, i, a.N);
    const Row8<DTY> ry = load_row8<DTY>(a.dY, base, i, a.N);
    float g[8], dx[8];
    load_vec8(a.gamma, a.dtw, i, a.N, 1.0f, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = (value<DTX>(rx, e) - mean) * rstd;
      dx[e] = rstd * (value<DTY>(ry, e) * g[e] - s1 - xh * s2);
    }
    store_row8<DTX>(a.dX, base, i, a.N, dx);
  }
}

// Their column sums: a workgroup takes 2048 columns of the rows parts apart.
template <int DTX, int DTY>
__global__ __launch_bounds__(256) void layer_norm_grad_columns_kernel(NormGradArgs a) {
  const uint32_t i = (blockIdx.x * 256u + threadIdx.x) * 8u;
  if (i >= a.N) return;
  float dg[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dg[e] = db[e] = 0.0f;
  for (uint32_t row = blockIdx.y; row < a.rows; row += a.parts) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    const Row8<DTX> rx = load_row8<DTX>(a.X, (size_t)row * a.N, i, a.N);
    const Row8<DTY> ry = load_row8<DTY>(a.dY, (size_t)row * a.N, i, a.N);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float dy = value<DTY>(ry, e);
      dg[e] = __builtin_fmaf(dy, (value<DTX>(rx, e) - mean) * rstd, dg[e]);
      db[e] += dy;
    }
  }
  float* const out = a.part + (size_t)blockIdx.y * 2u * a.N;
  store_row8<DT_F32>(out, 0, i, a.N, dg);
  store_row8<DT_F32>(out, a.N, i, a.N, db);
}

template <int DTX, int DTY, int T, int C>
inline void launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  note_launch("layer norm gradient, %d threads a row, %d values a thread, %u parts", T, 8 * C, a.parts);
  launch_kernel(layer_norm_grad_kernel<DTX, DTY, T, C>, dim3(a.parts), dim3(T > 256 ? T : 256), s, a);
}

template <int DTX, int DTY>
inline void launch_norm_grad_to(const NormGradArgs& a, hipStream_t s) {
  if (a.N > kNormLong) {
    launch_kernel(layer_norm_grad_long_kernel<DTX, DTY>, dim3(a.rows), dim3(1024), s, a);
    if (a.part)
      launch_kernel(layer_norm_grad_columns_kernel<DTX, DTY>, dim3((a.N + 2047u) / 2048u, a.parts), dim3(256), s, a);
    note_launch("layer norm gradient, long rows, %u parts", a.parts);
    return;
  }
  switch (norm_grad_threads(a.N)) {
    case 16: return launch_norm_grad<DTX, DTY, 16, 1>(a, s);
    case 64:
      if (a.N <= 512) return launch_norm_grad<DTX, DTY, 64, 1>(a, s);
      return launch_norm_grad<DTX, DTY, 64, 2>(a, s);
    case 256:
      if (a.N <= 2048) return launch_norm_grad<DTX, DTY, 256, 1>(a, s);
      return launch_norm_grad<DTX, DTY, 256, 2>(a, s);
    case 512: return launch_norm_grad<DTX, DTY, 512, 2>(a, s);
    default: return launch_norm_grad<DTX, DTY, 1024, 2>(a, s);
  }
}

template <int DTX>
inline int launch_layer_norm_grad(int dty, const NormGradArgs& a, hipStream_t s) {
  switch (dty) {
    case DT_F32: launch_norm_grad_to<DTX, DT_F32>(a, s); return 0;
    case DT_F16: launch_norm_grad_to<DTX, DT_F16>(a, s); return 0;
    case DT_BF16: launch_norm_grad_to<DTX, DT_BF16>(a, s); return 0;
    default: return -1;
  }
}

}  // namespace biasact
