// Products over groups of rows: the kernels' arguments, the lookup of a
// program's group from the device array of offsets, and the launchers.
//
// Group e is rows [start(e), end(e)) with start(e) = max over j <= e of
// off[j] and end(e) = start(e + 1), every offset clamped to [0, rows]: for
// any content of the array the groups are disjoint, in order and inside the
// operands.  A launch has one program per tile of an upper bound known on
// the host,
//   sum_e ceil(len(e) / BM) <= rows / BM + min(groups, rows),
// and each wavefront finds its own program's group from the offsets: 64
// groups per step, one per lane, by a prefix maximum (the starts) and a
// prefix sum (the tile counts).  No table, no second kernel, no host copy.
#pragma once
#include "launch.hpp"

namespace dg {

struct GroupedArgs {
    GemmArgs g;                // of group 0: M (RAGGED_M) and K (RAGGED_K) are set per group
    const int32_t *offsets;
    int32_t groups, rows;
    int64_t stride_bias;       // elements
    uint32_t tiles_n;          // output tiles along N
    uint32_t tiles;            // RAGGED_K: output tiles of one group
};

// Inclusive scans over the 64 lanes in six DPP steps: shifts by 1, 2, 4 and
// 8 inside each row of 16 lanes, then row 0's (2's) last value into row 1
// (3), then lane 31's into rows 2 and 3.  Lanes without a source take `id`.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int32_t dpp_or(int32_t id, int32_t v)
{
    return __builtin_amdgcn_update_dpp(id, v, CTRL, ROW_MASK, 0xf, false);
}

__device__ __forceinline__ int32_t wave_scan_max(int32_t v)    // v >= 0
{
    v = max(v, dpp_or<0x111, 0xf>(0, v));
    v = max(v, dpp_or<0x112, 0xf>(0, v));
    v = max(v, dpp_or<0x114, 0xf>(0, v));
    v = max(v, dpp_or<0x118, 0xf>(0, v));
    v = max(v, dpp_or<0x142, 0xa>(0, v));
    v = max(v, dpp_or<0x143, 0xc>(0, v));
    return v;
}

__device__ __forceinline__ int32_t wave_scan_add(int32_t v)
{
    v += dpp_or<0x111, 0xf>(0, v);
    v += dpp_or<0x112, 0xf>(0, v);
    v += dpp_or<0x114, 0xf>(0, v);
    v += dpp_or<0x118, 0xf>(0, v);
    v += dpp_or<0x142, 0xa>(0, v);
    v += dpp_or<0x143, 0xc>(0, v);
    return v;
}

__device__ __forceinline__ int32_t clamp_offset(int32_t v, int32_t rows)
{
    return v < 0 ? 0 : v > rows ? rows : v;
}

// 64 groups of the scan: lane l's group c * 64 + l, its rows and its tiles
// (0 past the last group).  `carry` is the largest offset so far.
struct GroupChunk {
    int32_t start, end;
    int32_t upto;             // inclusive prefix sum of the tiles, in this chunk
    int32_t tiles;
};

template <int BM>
__device__ __forceinline__ GroupChunk group_chunk(const int32_t *offsets, int32_t groups,
                                                  int32_t rows, int32_t c, int32_t &carry)
{
    const int lane = threadIdx.x & 63;
    const int32_t e = c * 64 + lane;
    const int32_t raw = e < groups ? clamp_offset(offsets[e + 1], rows) : 0;
    GroupChunk k;
    k.end = max(carry, wave_scan_max(raw));
    // the previous lane's end (wave_shr:1); lane 0 takes the carry
    k.start = __builtin_amdgcn_update_dpp(carry, k.end, 0x138, 0xf, 0xf, false);
    k.tiles = (int32_t)(((uint32_t)(k.end - k.start) + (BM - 1)) / BM);
    k.upto = wave_scan_add(k.tiles);
    carry = __builtin_amdgcn_readlane(k.end, 63);
    return k;
}

struct GroupTile {
    int32_t group;            // -1: the program has no tile
    int32_t start, rows;      // of the group
    uint32_t row_tile;        // inside the group
    uint32_t col_tile;
};

// Tile of program `pid` when every group's row tiles are BM rows and each
// row of tiles has tiles_n columns.  Programs are dealt to the 8 XCDs in
// contiguous runs of the tile order (as decode_program does), and inside a
// group the tiles walk bands of G tile rows column by column, so that the
// tiles running at one time on an XCD share few panels of A and B.
template <int BM, int G = 4>
__device__ __forceinline__ GroupTile find_group_tile(const int32_t *offsets, int32_t groups,
                                                     int32_t rows, uint32_t tiles_n, uint32_t pid)
{
    const int32_t chunks = (groups + 63) / 64;
    int32_t carry = clamp_offset(offsets[0], rows);
    const int32_t carry0 = carry;
    GroupChunk k = group_chunk<BM>(offsets, groups, rows, 0, carry);
    uint32_t total = (uint32_t)__builtin_amdgcn_readlane(k.upto, 63);
    for (int32_t c = 1; c < chunks; ++c) {
        k = group_chunk<BM>(offsets, groups, rows, c, carry);
        total += (uint32_t)__builtin_amdgcn_readlane(k.upto, 63);
    }
    GroupTile t{-1, 0, 0, 0, 0};
    const uint32_t P = total * tiles_n;      // at most the launch's grid, below 2^31
    if (pid >= P)
        return t;
    const uint32_t x = pid % kNumXcd, q = P / kNumXcd, r = P % kNumXcd;
    const uint32_t L = x * q + (x < r ? x : r) + pid / kNumXcd;
    // the group whose tiles hold L: its first tile row is `before`
    uint32_t before = 0;
    int32_t c = 0;
    if (chunks > 1) {
        carry = carry0;
        k = group_chunk<BM>(offsets, groups, rows, 0, carry);
    }
    for (;;) {
        const uint64_t past = __ballot((before + (uint32_t)k.upto) * tiles_n > L);
        if (past) {
            const int lane = __builtin_ctzll(past);
            const uint32_t own = (uint32_t)__builtin_amdgcn_readlane(k.tiles, lane);
            const uint32_t first = before + (uint32_t)__builtin_amdgcn_readlane(k.upto, lane) - own;
            const uint32_t in = L - first * tiles_n;           // inside the group
            const uint32_t band = in / (G * tiles_n), o = in - band * (G * tiles_n);
            const uint32_t left = own - band * G, h = left < G ? left : G;
            t.group = c * 64 + lane;
            t.start = __builtin_amdgcn_readlane(k.start, lane);
            t.rows = __builtin_amdgcn_readlane(k.end, lane) - t.start;
            t.col_tile = o / h;
            t.row_tile = band * G + (o - t.col_tile * h);
            return t;
        }
        before += (uint32_t)__builtin_amdgcn_readlane(k.upto, 63);
        ++c;                    // L < P: some chunk has the tile
        k = group_chunk<BM>(offsets, groups, rows, c, carry);
    }
}

// Rows of group e alone.
__device__ __forceinline__ void group_rows(const int32_t *offsets, int32_t rows, int32_t e,
                                           int32_t &start, int32_t &end)
{
    const int lane = threadIdx.x & 63;
    int32_t m = 0;
    for (int32_t j = lane; j <= e; j += 64)
        m = max(m, clamp_offset(offsets[j], rows));
    start = __builtin_amdgcn_readlane(wave_scan_max(m), 63);
    end = max(start, clamp_offset(offsets[e + 1], rows));
}

// The argument block of one group's product.
template <bool RAGGED_K>
__device__ __forceinline__ GemmArgs group_args(const GroupedArgs &a, int32_t e, int32_t start,
                                               int32_t len)
{
    const int64_t es = a.g.ab_type == DT_F32 ? 4 : 2, cs = a.g.c_type == DT_F32 ? 4 : 2;
    GemmArgs g = a.g;
    g.A = (const char *)g.A + (int64_t)start * g.lda * es;
    if (RAGGED_K) {
        g.K = len;
        g.B = (const char *)g.B + (int64_t)start * g.ldb * es;
        g.C = (char *)g.C + e * g.sc * cs;
        g.bias = nullptr;
        g.act = ACT_NONE;
    } else {
        g.M = len;
        g.B = (const char *)g.B + e * g.sb * es;
        g.C = (char *)g.C + (int64_t)start * g.ldc * cs;
        if (g.bias)
            g.bias = (const char *)g.bias + e * a.stride_bias * (g.bias_type == DT_F32 ? 4 : 2);
    }
    g.sa = g.sb = g.sc = 0;
    g.c_col = 0;
    g.write_partial = 0;
    return g;
}

struct QweightArgs {
    const void *A;
    const uint8_t *Q;
    const void *scales;
    const uint8_t *zeros;      // null: 8
    void *C;
    const void *bias;
    const int32_t *offsets;    // null: one group of M rows
    int32_t groups, rows;
    int64_t N, K, group_size;
    int64_t lda, ldc, ldq, lds;
    int64_t stride_q, stride_s, stride_bias;
    float alpha, beta;
    int32_t a_type, c_type, scale_type, bias_type, act;
    uint32_t tiles_n;
};

// Launchers; each returns hipSuccess or the launch error.
hipError_t launch_grouped_generic(const GroupedArgs &a, bool ragged_k, uint32_t programs,
                                  hipStream_t s);
// 16-bit matrix-core tiles (256 x 256 and 128 x 128)
hipError_t launch_grouped16_m256_bf16(const GroupedArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_grouped16_m256_f16(const GroupedArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_grouped16_m128(const GroupedArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_grouped16_k256(const GroupedArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_grouped16_k128(const GroupedArgs &a, uint32_t programs, hipStream_t s);
// fp32 matrix-core tile (128 x 128)
hipError_t launch_grouped_f32_m(const GroupedArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_grouped_f32_k(const GroupedArgs &a, uint32_t programs, hipStream_t s);
// few rows per group (kernel_stream.hip)
hipError_t launch_grouped_stream(int32_t variant, const GroupedArgs &a, uint32_t programs,
                                 hipStream_t s);
hipError_t launch_qweight_rows(int32_t variant, const QweightArgs &a, uint32_t programs,
                               hipStream_t s);
hipError_t launch_qweight_tile(const QweightArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_qweight_wide_tile(const QweightArgs &a, uint32_t programs, hipStream_t s);
hipError_t launch_qweight_generic(const QweightArgs &a, uint32_t programs, hipStream_t s);

constexpr int kGroupedGenericTile = 64;

} // namespace dg
