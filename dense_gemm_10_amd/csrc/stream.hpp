// Products of few rows of A with a large B: each weight is used once or a
// few times, so the kernels are bound by reading B from memory.  Shared by
// the grouped products (kernel_stream.hip) and the products with 4-bit
// weights (kernel_qstream.hip, kernel_qtile.hip).
//
// A workgroup owns 16 FM rows x 16 FN columns of one group's output and its
// KW wavefronts take the steps along K in turn (wavefront w: steps w, w +
// KW, ...), so that together they read consecutive memory.  B goes from
// memory straight into MFMA operand registers, with no LDS and no barrier
// in the loop; the next step's loads are issued before this step's MFMAs.
// A's rows come from the caches the same way (rows past the group's end
// repeat its last row and are not stored).  At the end the wavefronts'
// fp32 sums meet in LDS, are added in wavefront order (a fixed order: the
// result is reproducible) and take the epilogue once.
//
// Measured (MI355X): 64 rows on 64 groups, 2048 x 1024 bf16 36.4 us, 171 MB
// at 4.7 TB/s, what a large copy reaches; 1000 rows, 5 groups, 512 x 260
// fp32 9.2 us in a replayed graph (a fill of 64 floats there: 1.7): at most
// 180 workgroups, so that 76 of the 256 compute units idle, and each has 2.1
// MFLOP, 3.4 us of a unit's fp32 matrix rate; the rest is start, the latency
// of the few steps and the epilogue.
#pragma once
#include "grouped.hpp"
#include "mfma16.hpp"

namespace dg {

namespace {

// A load at a uniform base (scalar registers) plus a 32-bit byte offset per
// lane.  The base is kept as a pointer to global memory: from a plain pointer
// rebuilt out of scalar registers the compiler makes flat loads, whose two
// counters have to be waited for together, and the loads in flight are lost
// (one token through 16384 x 8192 4-bit weights: 34 us that way).
typedef const __attribute__((address_space(1))) char *global_base;

__device__ __forceinline__ global_base uniform_base(const void *p)
{
    return (global_base)(uintptr_t)uniform_i64((int64_t)(uintptr_t)p);
}

template <typename V>
__device__ __forceinline__ V load_at(global_base base, uint32_t offset)
{
    return *(const __attribute__((address_space(1))) V *)(base + offset);
}

__device__ __forceinline__ uint4 load16_at(global_base base, uint32_t offset)
{
    return __builtin_bit_cast(uint4, load_at<u32x4_nt>(base, offset));
}

// Sum the KW wavefronts' accumulators and store the tile.  Value v of lane
// l in block (i, j) is row 16 i + 4 (l / 16) + v and column col(j, l % 16)
// of the tile; `rows` x `cols` of the tile lie inside the output at (m0,
// n0) of g.C.
template <int FM, int FN, int KW, bool INTERLEAVED>
__device__ __forceinline__ void stream_store(const GemmArgs &g, int64_t m0, int64_t n0, int rows,
                                             int cols, const f32x4_t (&acc)[FM][FN], float *lds)
{
    constexpr int NT = 64 * KW, TILE = 16 * FM * 16 * FN;
    constexpr int LD = 16 * FN + 4;      // a 16-lane write's rows, 4 apart, on other banks
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float *mine = lds + wave * (16 * FM * LD);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = INTERLEAVED ? FN * (lane & 15) + j : 16 * j + (lane & 15);
                mine[(16 * i + 4 * (lane >> 4) + v) * LD + c] = acc[i][j][v];
            }
    lds_barrier();
    for (int o = tid; o < TILE; o += NT) {
        const int r = o / (16 * FN), c = o % (16 * FN);
        if (r >= rows || c >= cols)
            continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
            sum += lds[w * (16 * FM * LD) + r * LD + c];
        store_c(g, 0, m0 + r, n0 + c, epilogue_value(g, 0, m0 + r, n0 + c, sum));
    }
}

template <int FM, int FN, int KW>
constexpr size_t stream_lds_bytes() { return (size_t)KW * 16 * FM * (16 * FN + 4) * 4; }

} // namespace

} // namespace dg
