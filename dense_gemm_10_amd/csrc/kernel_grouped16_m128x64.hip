// Instantiations of the grouped 16-bit products (grouped16.hpp): ragged
// rows, 128 x 128 tile with
// 64-deep stages on 16 x 16 x 32 MFMAs.
#include "grouped16.hpp"

namespace dg {

hipError_t launch_grouped16_m128x64(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    return a.g.ab_type == DT_F16 ? launch_grouped_m<DT_F16, 128, 128, 2, 64, 16>(a, programs, s)
                                 : launch_grouped_m<DT_BF16, 128, 128, 2, 64, 16>(a, programs, s);
}

} // namespace dg
