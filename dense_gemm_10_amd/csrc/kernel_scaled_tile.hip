// 8-bit products on the tiles of mfma16.hpp: rows on 16 bytes, K a whole
// number of pairs.  Everything up to the MFMA sees 16-bit elements, two
// integers each.
#include "grouped16.hpp"
#include "scaled.hpp"

namespace dg {

namespace {

// Leading dimensions and K in pairs.
__device__ __forceinline__ GemmArgs in_pairs(GemmArgs g)
{
    g.lda >>= 1;
    g.ldb >>= 1;
    g.K >>= 1;
    g.c_col = 0;
    g.write_partial = 0;
    return g;
}

template <int BM, int BN, int NS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(mfma16_per_cu(BM, BN, NS, 64))))
void scaled_tile_kernel(ScaledArgs a)
{
    extern __shared__ uint4 lds[];
    const GroupTile t = scaled_tile<BM>(a);
    if (t.group < 0)
        return;
    const GemmArgs g = in_pairs(scaled_args(a, t.group, t.start, t.rows));
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    const RowColScales sc{row_scales(a, t.start), col_scales(a, t.group), a.scale_type};
    mfma16_tile<DT_I8, BM, BN, 2, 2, NS, 64, false, false, 16>(g, tc, 0, g.K, nullptr, lds, sc);
}

template <int BM, int BN, int NS>
hipError_t launch(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    hipLaunchKernelGGL((scaled_tile_kernel<BM, BN, NS>), dim3(programs), dim3(256),
                       (size_t)mfma16_lds_bytes(BM, BN, NS, 64, 16), s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_scaled_tile(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    switch (variant) {
    case 0: return launch<128, 128, 2>(a, programs, s);
    case 1: return launch<128, 256, 3>(a, programs, s);
    case 2: return launch<256, 256, 2>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
