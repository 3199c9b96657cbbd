// Grouped products, int8 (one scale a row of A and of B).
#include "grouped.hpp"

namespace qgemm {
hipError_t launch_grouped_i8(int tile, bool bias, const GroupedParams &p, hipStream_t s)
{
    return bias ? launch_grouped_tile<PATH_I8, true>(tile, p, s) : launch_grouped_tile<PATH_I8, false>(tile, p, s);
}
}  // namespace qgemm
