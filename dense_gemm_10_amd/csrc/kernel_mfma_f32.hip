// fp32 GEMM on the matrix cores: the kernel around the tile of mfma_f32.hpp
// and its launcher.
#include "mfma_f32.hpp"

namespace dg {

namespace {

template <int BM, int BN, int WM, int WN, int FBK, bool A_COL, bool B_COL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_mfma_f32_kernel(GemmArgs g)
{
    extern __shared__ float smem[];
    const TileCoord tc = decode_program(blockIdx.x, g.sched);
    int64_t kb, ke;
    split_range(g, tc.s, kb, ke);
    mfma_f32_tile<BM, BN, WM, WN, FBK, A_COL, B_COL>(g, tc, kb, ke, smem);
}

template <int BM, int BN, int WM, int WN, int FBK>
hipError_t launch_f32(const GemmArgs &g, const Plan &p, hipStream_t stream)
{
    const size_t lds = f32_lds_bytes<BM, BN, WM, WN, FBK>();
    dim3 grid((unsigned)p.programs), block(64 * WM * WN);
    if (!g.a_col && !g.b_col)
        hipLaunchKernelGGL((gemm_mfma_f32_kernel<BM, BN, WM, WN, FBK, false, false>), grid, block, lds,
                           stream, g);
    else if (!g.a_col && g.b_col)
        hipLaunchKernelGGL((gemm_mfma_f32_kernel<BM, BN, WM, WN, FBK, false, true>), grid, block, lds,
                           stream, g);
    else if (g.a_col && !g.b_col)
        hipLaunchKernelGGL((gemm_mfma_f32_kernel<BM, BN, WM, WN, FBK, true, false>), grid, block, lds,
                           stream, g);
    else
        hipLaunchKernelGGL((gemm_mfma_f32_kernel<BM, BN, WM, WN, FBK, true, true>), grid, block, lds,
                           stream, g);
    return hipGetLastError();
}

} // namespace

// Entries 0 and 1 are the large and small tiles of the automatic choice;
// the 32-deep ones are selectable by name and by the tuned table.
hipError_t launch_mfma_f32(const GemmArgs &g, const Plan &p, hipStream_t stream)
{
    switch (p.tile.variant) {
    case 0: return launch_f32<256, 256, 2, 2, 16>(g, p, stream);
    case 1: return launch_f32<128, 128, 2, 2, 16>(g, p, stream);
    case 2: return launch_f32<256, 256, 2, 2, 32>(g, p, stream);
    case 3: return launch_f32<128, 128, 2, 2, 32>(g, p, stream);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
