// Grouped products of 16-bit operands on the matrix cores: the tile code of
// mfma16.hpp run on one group's product per workgroup.  Instantiated by the
// kernel_grouped16_*.hip files.
//
// A group's first row is a whole number of leading dimensions from the
// operand's start, and leading dimensions are multiples of 8 elements, so
// every group's rows start on 16 bytes and the tile's DMA, swizzle and
// masks serve a group exactly as they serve a matrix: RAGGED_M masks the
// rows past the group's end (they may be another group's), RAGGED_K ends
// the K loop at the group's last row with the partial K tile that masks K.
#pragma once
#include "grouped.hpp"
#include "mfma16.hpp"

namespace dg {

namespace {

// RAGGED_M: A row-major, B[e] K-contiguous (BT false) or N-contiguous.
template <int T, int BM, int BN, int NS, int BK, bool BT, int MS>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(mfma16_per_cu(BM, BN, NS, BK))))
void grouped_m_kernel(GroupedArgs a)
{
    extern __shared__ uint4 lds[];
    const GroupTile t = find_group_tile<BM>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
    if (t.group < 0)
        return;
    const GemmArgs g = group_args<false>(a, t.group, t.start, t.rows);
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    mfma16_tile<T, BM, BN, 2, 2, NS, BK, false, BT, MS>(g, tc, 0, g.K, nullptr, lds);
}

// RAGGED_K: both operands with their rows along K (A M-contiguous, B
// N-contiguous), so both go through the transposing LDS reads.  Programs
// are dealt to the XCDs in contiguous runs of (group, tile): the tiles of
// one group, which share its rows of A and B, run on one XCD.
template <int T, int BM, int BN, int NS, int BK, int MS>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(mfma16_per_cu(BM, BN, NS, BK))))
void grouped_k_kernel(GroupedArgs a)
{
    extern __shared__ uint4 lds[];
    const uint32_t P = gridDim.x, x = blockIdx.x % kNumXcd, r = P % kNumXcd;
    const uint32_t L = x * (P / kNumXcd) + (x < r ? x : r) + blockIdx.x / kNumXcd;
    const uint32_t e = L / a.tiles, t = L - e * a.tiles;
    int32_t start, end;
    group_rows(a.offsets, a.rows, (int32_t)e, start, end);
    const GemmArgs g = group_args<true>(a, (int32_t)e, start, end - start);
    const uint32_t tm = t / a.tiles_n;
    const TileCoord tc{0, 0, (int32_t)tm, (int32_t)(t - tm * a.tiles_n)};
    mfma16_tile<T, BM, BN, 2, 2, NS, BK, true, true, MS>(g, tc, 0, g.K, nullptr, lds);
}

template <int T, int BM, int BN, int NS, int BK, int MS>
hipError_t launch_grouped_m(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr size_t lds = (size_t)mfma16_lds_bytes(BM, BN, NS, BK, MS);
    if (a.g.b_col)
        hipLaunchKernelGGL((grouped_m_kernel<T, BM, BN, NS, BK, false, MS>), dim3(programs),
                           dim3(256), lds, s, a);
    else
        hipLaunchKernelGGL((grouped_m_kernel<T, BM, BN, NS, BK, true, MS>), dim3(programs),
                           dim3(256), lds, s, a);
    return hipGetLastError();
}

template <int T, int BM, int BN, int NS, int BK, int MS>
hipError_t launch_grouped_k(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    hipLaunchKernelGGL((grouped_k_kernel<T, BM, BN, NS, BK, MS>), dim3(programs), dim3(256),
                       (size_t)mfma16_lds_bytes(BM, BN, NS, BK, MS), s, a);
    return hipGetLastError();
}

} // namespace

} // namespace dg
