// grouped.hpp -- grouped products: the host's choice of tile and the launch of
// one path's kernels.
#pragma once
#include "../qgemm_launch.hpp"
#include "experts.hpp"

namespace qgemm {

// Per-path entry points, one translation unit each.
hipError_t launch_grouped_i8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_f8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_f8b(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_mx8(int tile, bool bias, const GroupedParams &p, hipStream_t s);
hipError_t launch_grouped_mx4(int tile, bool bias, const GroupedParams &p, hipStream_t s);

template <int PATH, bool BIAS>
hipError_t launch_grouped_tile(int tile, const GroupedParams &p, hipStream_t s)
{
    constexpr int BROWS = PATH == PATH_F8B ? 128 : 1;
    const dim3 grid((unsigned)((int64_t)p.tiles_m * p.tiles_n)), block(tile_threads(tile));
    switch (tile) {
    case SKINNY16_TILE:
        hipLaunchKernelGGL((qgemm_skinny_kernel<PATH, 1, skinny_depth<PATH, 1>(), BIAS, BROWS, true>), grid, block, 0, s,
                           p);
        break;
    case DMA128_TILE:
        hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 2, 2, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s, p);
        break;
    case DMA8_TILE:
        if constexpr (PATH != PATH_F8B) {
            hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 4, 4, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s,
                               p);
            break;
        }
        return hipErrorInvalidValue;
    case F8B256_TILE:
        if constexpr (PATH == PATH_F8B) {
            hipLaunchKernelGGL((qgemm_dma_kernel<PATH, 2, 4, 2, BIAS, BROWS, OUT_BF16, false, true>), grid, block, 0, s,
                               p);
            break;
        }
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace qgemm
