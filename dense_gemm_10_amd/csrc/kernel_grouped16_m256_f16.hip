// Instantiations of the grouped 16-bit products (grouped16.hpp): f16, ragged
// rows, 256 x 256 tile.
#include "grouped16.hpp"

namespace dg {

hipError_t launch_grouped16_m256_f16(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    return launch_grouped_mixed<DT_F16>(a, programs, s);
}

} // namespace dg
