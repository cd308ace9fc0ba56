// gemm_mx_launch.hpp — choice of the kernel for a product with an MXFP4 B.
#pragma once

#include "gemm_mx.hpp"
#include "gemm_mx_tile.hpp"

namespace biasact {

inline uint64_t tiles_of(const MxGemmArgs& a, uint32_t bm, uint32_t bn) {
  return (uint64_t)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn);
}

// Streaming kernel of 16 MB rows of A.  Its workgroups take the 256 CUs in
// rounds, and a round's time goes with the rows that a workgroup loads per
// group of k: NB blocks of codes, MB blocks of A (four times the bytes when A is
// 16-bit), and about two blocks' worth for what does not depend on them.
template <int DTA, int DTO, int MB>
inline void launch_mx_stream_nb(const MxGemmArgs& a, hipStream_t s) {
  auto cost = [&](uint32_t nb) {
    return (tiles_of(a, 16 * MB, 16 * nb) + 255) / 256 * (nb + (DTA == DT_MXFP4 ? 1 : 4) * MB + 2);
  };
  const uint64_t c1 = cost(1), c2 = cost(2);
  if constexpr (DTA != DT_F16 || MB < 4) {            // (fp16's second way leaves no registers for 4 x 4)
    const uint64_t c4 = cost(4);
    if (c4 <= c2 && c4 <= c1) return launch_mx_stream<DTA, DTO, 4, MB>(a, s);
  }
  if (c2 <= c1) launch_mx_stream<DTA, DTO, 2, MB>(a, s);
  else launch_mx_stream<DTA, DTO, 1, MB>(a, s);
}

template <int DTA, int DTO>
inline void launch_gemm_mx_to(const MxGemmArgs& a, hipStream_t s) {
  if (a.K < (DTA == DT_MXFP4 ? 1u : 8u)) return launch_mx_short<DTA, DTO>(a, s);
  if constexpr (DTA == DT_MXFP4) {
    // Past one round of 64x64 blocks the tiled kernels are faster, but for two
    // rounds over a long k, where 128x128 tiles leave half of the CUs idle (us,
    // streaming and 128x128: 512x4096x4096 15.2 and 12.6, x6144 20.9 and 17.8, x8192
    // 25.4 and 27.6, x16384 41.8 and 49.9; 192x8192x12288 32.0 and 38.2; three
    // rounds, 700x4096x12288, 48.3 and 38.0; one round, 64x16384x4096, 9.9 and 15.9).
    // Between the tiles their rounds decide, at K = 4096: up to 256 of 128x128 15 us,
    // 512 of them 24, 256 of 256x256 40.  E.g. 6464x790x7221: 44.5 with 128x128, 54.8
    // with 256x256; 4096^3: 52.6 and 40.2.
    const uint64_t blocks = tiles_of(a, 64, 64);
    if (blocks > (a.G < 64 ? 256 : 512)) {
      const uint64_t t128 = tiles_of(a, 128, 128);
      const uint64_t small = t128 <= 256 ? 15 : (t128 + 511) / 512 * 24, large = (tiles_of(a, 256, 256) + 255) / 256 * 40;
      if (large < small) return launch_mx_tile<DTO, 2, 4, 4, 2>(a, s);
      return launch_mx_tile<DTO, 2, 2, 2, 2>(a, s);
    }
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
