// Grouped products, e4m3 (one scale a row of A and of B).
#include "grouped.hpp"

namespace qgemm {
hipError_t launch_grouped_f8(int tile, bool bias, const GroupedParams &p, hipStream_t s)
{
    return bias ? launch_grouped_tile<PATH_F8, true>(tile, p, s) : launch_grouped_tile<PATH_F8, false>(tile, p, s);
}
}  // namespace qgemm
