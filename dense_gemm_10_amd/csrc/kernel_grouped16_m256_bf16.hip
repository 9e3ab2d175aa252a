// Instantiations of the grouped 16-bit products (grouped16.hpp): bf16, ragged
// rows, 256 x 256 tile.
#include "grouped16.hpp"

namespace dg {

hipError_t launch_grouped16_m256_bf16(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    return launch_grouped_mixed<DT_BF16>(a, programs, s);
}

} // namespace dg
