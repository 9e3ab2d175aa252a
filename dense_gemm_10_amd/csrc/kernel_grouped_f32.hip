// Grouped fp32 products on the matrix cores: the 128 x 128 tile of
// mfma_f32.hpp run on one group's product per workgroup (as grouped16.hpp
// does with the 16-bit tile).
#include "grouped.hpp"
#include "mfma_f32.hpp"

namespace dg {

namespace {

constexpr int FT = 128, FK = 16;

template <bool B_COL>
__global__ __launch_bounds__(256) void grouped_f32_m_kernel(GroupedArgs a)
{
    extern __shared__ float smem[];
    const GroupTile t = find_group_tile<FT>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
    if (t.group < 0)
        return;
    const GemmArgs g = group_args<false>(a, t.group, t.start, t.rows);
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    mfma_f32_tile<FT, FT, 2, 2, FK, false, B_COL, true>(g, tc, 0, g.K, smem);
}

__global__ __launch_bounds__(256) void grouped_f32_k_kernel(GroupedArgs a)
{
    extern __shared__ float smem[];
    const uint32_t e = blockIdx.x / a.tiles, t = blockIdx.x - e * a.tiles, tm = t / a.tiles_n;
    int32_t start, end;
    group_rows(a.offsets, a.rows, (int32_t)e, start, end);
    const GemmArgs g = group_args<true>(a, (int32_t)e, start, end - start);
    const TileCoord tc{0, 0, (int32_t)tm, (int32_t)(t - tm * a.tiles_n)};
    mfma_f32_tile<FT, FT, 2, 2, FK, true, false>(g, tc, 0, g.K, smem);
}

} // namespace

hipError_t launch_grouped_f32_m(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr size_t lds = f32_lds_bytes<FT, FT, 2, 2, FK>();
    if (a.g.b_col)
        hipLaunchKernelGGL(grouped_f32_m_kernel<true>, dim3(programs), dim3(256), lds, s, a);
    else
        hipLaunchKernelGGL(grouped_f32_m_kernel<false>, dim3(programs), dim3(256), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_grouped_f32_k(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    hipLaunchKernelGGL(grouped_f32_k_kernel, dim3(programs), dim3(256),
                       (f32_lds_bytes<FT, FT, 2, 2, FK>()), s, a);
    return hipGetLastError();
}

} // namespace dg
