// Stand-ins for the launchers of the grouped and 4-bit-weight kernels, linked
// into the host-code sanitizer build of the library
// (tests/test_grouped_sanitizers.py) in place of the kernels.  Nothing in
// that test launches a kernel; each stand-in reports a launch error if it is
// ever reached.
#include "grouped.hpp"

namespace dg {

#define STUB(name) \
    hipError_t name(const GroupedArgs &, uint32_t, hipStream_t) { return hipErrorInvalidValue; }
STUB(launch_grouped16_m256_bf16)
STUB(launch_grouped16_m256_f16)
STUB(launch_grouped16_m128)
STUB(launch_grouped16_k256)
STUB(launch_grouped16_k128)
STUB(launch_grouped_f32_m)
STUB(launch_grouped_f32_k)
hipError_t launch_grouped_stream(int32_t, const GroupedArgs &, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_grouped_generic(const GroupedArgs &, bool, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_qweight_rows(int32_t, const QweightArgs &, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_qweight_tile(const QweightArgs &, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_qweight_wide_tile(const QweightArgs &, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_qweight_generic(const QweightArgs &, uint32_t, hipStream_t)
{
    return hipErrorInvalidValue;
}

} // namespace dg
