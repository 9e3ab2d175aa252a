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
//
// Measured (MI355X, bf16): ragged rows, 8192 rows, 16 groups of 0.5 to 1.5
// times the mean, 4096 x 4096, bias and GELU: 337 us, 0.82 PFLOP/s; matrix
// pipe and the workgroups of the last, partly filled pass bound it.  Ragged
// K, 8192 rows, 16 groups, 2048 x 2048 into fp32: 96-106 us, 268 MB of C
// written (3.2-3.5 TB/s of all traffic).
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

// RAGGED_M on 256 x 256 tiles, with half-height ones where they save a wave.
// A group's last tile is 128 rows high if 128 hold its rows, and the whole
// tiles that would start a last, partly filled wave of the chip's 256
// compute units are cut into two halves each if those and the short tiles
// fit into one wave together.  Whole tiles come first.  A half tile takes
// 0.6 of a whole one's time (it has half the matrix work per byte staged, in
// a deeper ring), so 2.5 waves of whole tiles, run as 3, become 2.6.
struct MixedTile {
    int32_t group;            // -1: none
    int32_t start, rows;
    bool half;
    uint32_t row_tile;        // in 256 rows, or in 128 if half
    uint32_t col_tile;
};

struct MixedChunk {
    GroupChunk k;             // .tiles, .upto: whole tiles
    int32_t halves, halves_upto;
};

__device__ __forceinline__ MixedChunk mixed_chunk(const int32_t *offsets, int32_t groups, int32_t rows,
                                                  int32_t c, int32_t &carry)
{
    MixedChunk m;
    m.k = group_chunk<256>(offsets, groups, rows, c, carry);
    const int32_t rem = (m.k.end - m.k.start) & 255;
    m.halves = rem > 0 && rem <= 128;
    m.k.tiles -= m.halves;
    m.halves_upto = wave_scan_add(m.halves);
    m.k.upto -= m.halves_upto;
    return m;
}

__device__ __forceinline__ MixedTile find_mixed_tile(const int32_t *offsets, int32_t groups, int32_t rows,
                                                     uint32_t tiles_n, uint32_t pid)
{
    const int32_t chunks = (groups + 63) / 64, carry0 = clamp_offset(offsets[0], rows);
    int32_t carry = carry0;
    MixedChunk m = mixed_chunk(offsets, groups, rows, 0, carry);
    uint32_t whole = (uint32_t)__builtin_amdgcn_readlane(m.k.upto, 63);
    uint32_t halves = (uint32_t)__builtin_amdgcn_readlane(m.halves_upto, 63);
    for (int32_t c = 1; c < chunks; ++c) {
        m = mixed_chunk(offsets, groups, rows, c, carry);
        whole += (uint32_t)__builtin_amdgcn_readlane(m.k.upto, 63);
        halves += (uint32_t)__builtin_amdgcn_readlane(m.halves_upto, 63);
    }
    MixedTile t{-1, 0, 0, false, 0, 0};
    constexpr uint32_t W = 256;                   // compute units: workgroups of a wave
    uint32_t cut = whole * tiles_n % W;           // whole tiles of the last wave
    if (2 * cut + halves * tiles_n > W)
        cut = 0;
    const uint32_t kept = whole * tiles_n - cut, small = 2 * cut + halves * tiles_n;
    if (pid >= kept + small)
        return t;
    // the tile's index among the whole ones, or its group's among the halves
    auto remap = [](uint32_t i, uint32_t n) {     // contiguous runs to the XCDs
        const uint32_t x = i % kNumXcd, r = n % kNumXcd;
        return x * (n / kNumXcd) + (x < r ? x : r) + i / kNumXcd;
    };
    uint32_t index, lower = 0;
    bool of_whole = true;
    if (pid < kept) {
        index = remap(pid, kept);
    } else {
        const uint32_t i = remap(pid - kept, small);
        t.half = true;
        of_whole = i < 2 * cut;
        index = of_whole ? kept + i / 2 : i - 2 * cut;
        lower = of_whole ? i % 2 : 0;
    }
    uint32_t before = 0;
    if (chunks > 1) {
        carry = carry0;
        m = mixed_chunk(offsets, groups, rows, 0, carry);
    }
    for (int32_t c = 0;;) {
        const int32_t upto = of_whole ? m.k.upto : m.halves_upto;
        const uint64_t past = __ballot((before + (uint32_t)upto) * tiles_n > index);
        if (past) {
            const int lane = __builtin_ctzll(past);
            const uint32_t own =
                (uint32_t)__builtin_amdgcn_readlane(of_whole ? m.k.tiles : m.halves, lane);
            const uint32_t first = before + (uint32_t)__builtin_amdgcn_readlane(upto, lane) - own;
            const uint32_t in = index - first * tiles_n;
            const uint32_t band = in / (4 * tiles_n), o = in - band * (4 * tiles_n);
            const uint32_t left = own - band * 4, h = left < 4 ? left : 4;
            t.group = c * 64 + lane;
            t.start = __builtin_amdgcn_readlane(m.k.start, lane);
            t.rows = __builtin_amdgcn_readlane(m.k.end, lane) - t.start;
            t.col_tile = o / h;
            const uint32_t row = band * 4 + (o - t.col_tile * h);
            t.row_tile = !of_whole ? (uint32_t)t.rows / 256 * 2 : t.half ? 2 * row + lower : row;
            return t;
        }
        before += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
        ++c;                    // some chunk has the tile
        m = mixed_chunk(offsets, groups, rows, c, carry);
    }
}

template <int T, bool BT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1)))
void grouped_m_mixed_kernel(GroupedArgs a)
{
    extern __shared__ uint4 lds[];
    const MixedTile t = find_mixed_tile(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
    if (t.group < 0)
        return;
    const GemmArgs g = group_args<false>(a, t.group, t.start, t.rows);
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    if (!t.half)
        mfma16_tile<T, 256, 256, 2, 2, 2, 64, false, BT, 16>(g, tc, 0, g.K, nullptr, lds);
    else                                          // never empty: a whole tile has more than 128 rows
        mfma16_tile<T, 128, 256, 2, 2, 3, 64, false, BT, 16>(g, tc, 0, g.K, nullptr, lds);
}

template <int T>
hipError_t launch_grouped_mixed(const GroupedArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr int l0 = mfma16_lds_bytes(256, 256, 2, 64, 16), l1 = mfma16_lds_bytes(128, 256, 3, 64, 16);
    constexpr size_t lds = l0 > l1 ? l0 : l1;
    // a wave's tail cut in halves adds at most half a wave of programs
    const dim3 grid(programs + 128);
    if (a.g.b_col)
        hipLaunchKernelGGL((grouped_m_mixed_kernel<T, false>), grid, dim3(256), lds, s, a);
    else
        hipLaunchKernelGGL((grouped_m_mixed_kernel<T, true>), grid, dim3(256), lds, s, a);
    return hipGetLastError();
}

// RAGGED_K: both operands with their rows along K (A M-contiguous, B
// N-contiguous), so both go through the transposing LDS reads.
//
// Order of the (group, tile) programs.  The 8 XCDs take runs of S of them in
// turn, so that each gets an eighth of every group's work: in one long run
// per XCD the XCD with the longest groups finishes last (8 groups of 4096 x
// 4096 over 16384 rows, lengths from 0.5 to 1.5 of the mean: 918 us, 521 in
// runs of 16; groups of one length 541 and 516).  Inside a group the tiles
// walk bands of 4 tile rows column by column: a run of 32 reads 4 panels of
// A and 8 of B.
template <int S>
__device__ __forceinline__ uint32_t dealt_in_runs(uint32_t pid, uint32_t programs)
{
    const uint32_t whole = programs / (S * kNumXcd) * (S * kNumXcd);
    if (pid < whole) {
        const uint32_t x = pid % kNumXcd, i = pid / kNumXcd;
        return (i / S * kNumXcd + x) * S + i % S;
    }
    const uint32_t n = programs - whole, i = pid - whole, x = i % kNumXcd, r = n % kNumXcd;
    return whole + x * (n / kNumXcd) + (x < r ? x : r) + i / kNumXcd;
}

template <int T, int BM, int BN, int NS, int BK, int MS>
__global__ __launch_bounds__(256)
__attribute__((amdgpu_waves_per_eu(mfma16_per_cu(BM, BN, NS, BK))))
void grouped_k_kernel(GroupedArgs a)
{
    extern __shared__ uint4 lds[];
    constexpr uint32_t G = 4;
    const uint32_t L = dealt_in_runs<BM * BN >= 256 * 256 ? 16 : 32>(blockIdx.x, gridDim.x);
    const uint32_t e = L / a.tiles, t = L - e * a.tiles;
    int32_t start, end;
    group_rows(a.offsets, a.rows, (int32_t)e, start, end);
    const GemmArgs g = group_args<true>(a, (int32_t)e, start, end - start);
    const uint32_t band = t / (G * a.tiles_n), o = t - band * (G * a.tiles_n);
    const uint32_t left = a.tiles / a.tiles_n - band * G, h = left < G ? left : G;
    const TileCoord tc{0, 0, (int32_t)(band * G + o % h), (int32_t)(o / h)};
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
