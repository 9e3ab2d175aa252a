// Instantiations of the grouped 16-bit products (grouped16.hpp): ragged K,
// 128 x 128 tile.
#include "grouped16.hpp"

namespace dg {

// A ring of four stages hides more latency where a CU has one or two
// workgroups, a ring of two lets it hold four, whose stores and loads then
// overlap (us, bf16, fp32 out): 8 groups of 256 x 256, 8192 rows 17 on four
// stages, 32 on two; 32 of 512 x 512, 4096 rows 11.4 and 12.9; 16 of 1024 x
// 1024, 8192 rows 33.5 and 32.6; 16 of 2048 x 2048, 8192 rows 119 and 102;
// 4 of 4096 x 4096, 512 rows 65 and 50.
hipError_t launch_grouped16_k128(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    const bool f16 = a.g.ab_type == DT_F16;
    if (programs >= 1024)
        return f16 ? launch_grouped_k<DT_F16, 128, 128, 2, 32, 32>(a, programs, s)
                   : launch_grouped_k<DT_BF16, 128, 128, 2, 32, 32>(a, programs, s);
    return f16 ? launch_grouped_k<DT_F16, 128, 128, 4, 32, 32>(a, programs, s)
               : launch_grouped_k<DT_BF16, 128, 128, 4, 32, 32>(a, programs, s);
}

} // namespace dg
