// gemm_mx_launch.hpp — choice of the kernel for a product with an MXFP4 B.
#pragma once

#include "gemm_mx.hpp"
#include "gemm_mx_tile.hpp"

namespace biasact {

template <int DTA, int DTO, int MB>
inline void launch_mx_stream_nb(const MxGemmArgs& a, hipStream_t s) {
  // the widest block of B that still gives every CU a workgroup
  const uint64_t tm = (a.M + 16 * MB - 1) / (16 * MB);
  auto tiles = [&](uint32_t nb) { return tm * ((a.N + 16 * nb - 1) / (16 * nb)); };
  if (tiles(4) >= 256) launch_mx_stream<DTA, DTO, 4, MB, 8>(a, s);
  else if (tiles(2) >= 256) launch_mx_stream<DTA, DTO, 2, MB, 8>(a, s);
  else launch_mx_stream<DTA, DTO, 1, MB, 8>(a, s);
}

template <int DTA, int DTO>
inline void launch_gemm_mx_to(const MxGemmArgs& a, hipStream_t s) {
  if (a.K < (DTA == DT_MXFP4 ? 1u : 8u)) return launch_mx_short<DTA, DTO>(a, s);
  if constexpr (DTA == DT_MXFP4) {
    const uint64_t tiles = (uint64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
    if (tiles >= 64) return launch_mx_tile<DTO, 4, 2>(a, s);
  }
  if (a.M <= 16) launch_mx_stream_nb<DTA, DTO, 1>(a, s);
  else if (a.M <= 32) launch_mx_stream_nb<DTA, DTO, 2>(a, s);
  else launch_mx_stream_nb<DTA, DTO, 4>(a, s);
}

template <int DTA>
inline int launch_gemm_mx(int dto, const MxGemmArgs& a, hipStream_t s) {
  switch (dto) {
    case DT_F32: launch_gemm_mx_to<DTA, DT_F32>(a, s); return 0;
    case DT_F16: launch_gemm_mx_to<DTA, DT_F16>(a, s); return 0;
    case DT_BF16: launch_gemm_mx_to<DTA, DT_BF16>(a, s); return 0;
    default: return -1;
  }
}

}  // namespace biasact
