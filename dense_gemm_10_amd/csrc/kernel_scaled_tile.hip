// 8-bit products on the tiles of mfma16.hpp: rows on 16 bytes, K a whole
// number of pairs.  Everything up to the MFMA sees 16-bit elements, two
// integers each.
//
// Measured (MI355X, bf16 out, codes uniform in +-127): 16384^3 2.68 POP/s, 8192^3
// 2.77, 4096^3 2.42 (57 us in the steady state; 63 to 66 in the first calls).
// Fitted over K in the steady state, a whole 256 x 256 tile takes 1.4 us a stage
// of 128 bytes and 11.5 us beside its stages (16 with the tanh GELU, 18.7 with
// the erf form), a 128 x 256 half 0.8 and 9 (10.5 and 12).  The matrix pipe is
// busy 64 % of the cycles at 2.0 GHz, without bank conflicts; 61 % in the 16-bit
// kernel of the same bytes.  8192 rows, 16 groups, 4096 x 4096 157 us, with bias
// and erf GELU 176, and 178 to 195 in a trace of single calls.
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

// Eight wavefronts share a tile, two on a SIMD: one's waits are the other's
// matrix work, and a wavefront's sums, at most 128 registers, stay among the
// 256 that vector instructions read.  With four wavefronts and sums in both
// halves of the register file the compiler copies them back and forth in the
// K loop (8192 rows, 16 groups, 4096 x 4096: 260 us a call, 203 with the
// copies suppressed), and without the copies one wavefront per SIMD was still
// an eighth slower (4096 x 4096 x 4096, 62 us against 54 in the one run that
// had both; this kernel's steady time is 57).
template <int BM, int BN, int NS>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
void scaled_tile_kernel(ScaledArgs a)
{
    extern __shared__ uint4 lds[];
    const GroupTile t = scaled_tile<BM>(a);
    if (t.group < 0)
        return;
    const GemmArgs g = in_pairs(scaled_args(a, t.group, t.start, t.rows));
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    const RowColScales sc{row_scales(a, t.start), col_scales(a, t.group), a.scale_type};
    mfma16_tile<DT_I8, BM, BN, 2, 4, NS, 64, false, false, 16>(g, tc, 0, g.K, nullptr, lds, sc);
}

// 256 x 256 tiles with half-height ones where they save a wave, as
// find_mixed_tile deals them; of one matrix without offsets, the same deal.
__device__ __forceinline__ MixedTile matrix_mixed_tile(int32_t rows, uint32_t tiles_n, uint32_t pid)
{
    constexpr uint32_t W = 256;                   // compute units
    const uint32_t rem = (uint32_t)rows & 255, last = rem > 0 && rem <= 128;   // a half tile at the end
    const uint32_t own = ((uint32_t)rows + 255) / 256 - last;
    uint32_t cut = own * tiles_n % W;
    if (2 * cut + last * tiles_n > W)
        cut = 0;
    const uint32_t kept = own * tiles_n - cut, small = 2 * cut + last * tiles_n;
    MixedTile t{-1, 0, 0, false, 0, 0};
    if (pid >= kept + small)
        return t;
    auto remap = [](uint32_t i, uint32_t n) {     // contiguous runs to the XCDs
        const uint32_t x = i % kNumXcd, r = n % kNumXcd;
        return x * (n / kNumXcd) + (x < r ? x : r) + i / kNumXcd;
    };
    uint32_t index, lower = 0;
    if (pid < kept) {
        index = remap(pid, kept);
    } else {
        const uint32_t i = remap(pid - kept, small);
        t.half = true;
        index = kept + i / 2;
        lower = i % 2;
        if (i >= 2 * cut) {                       // the last rows' half tiles
            t.group = 0;
            t.rows = rows;
            t.row_tile = (uint32_t)rows / 256 * 2;
            t.col_tile = i - 2 * cut;
            return t;
        }
    }
    const uint32_t band = index / (4 * tiles_n), o = index - band * (4 * tiles_n);
    const uint32_t left = own - band * 4, h = left < 4 ? left : 4;
    t.group = 0;
    t.rows = rows;
    t.col_tile = o / h;
    const uint32_t row = band * 4 + (o - t.col_tile * h);
    t.row_tile = t.half ? 2 * row + lower : row;
    return t;
}

__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
void scaled_mixed_kernel(ScaledArgs a)
{
    extern __shared__ uint4 lds[];
    const MixedTile t = a.offsets ? find_mixed_tile(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x)
                                  : matrix_mixed_tile(a.rows, a.tiles_n, blockIdx.x);
    if (t.group < 0)
        return;
    const GemmArgs g = in_pairs(scaled_args(a, t.group, t.start, t.rows));
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    const RowColScales sc{row_scales(a, t.start), col_scales(a, t.group), a.scale_type};
    if (!t.half)
        mfma16_tile<DT_I8, 256, 256, 2, 4, 2, 64, false, false, 16>(g, tc, 0, g.K, nullptr, lds, sc);
    else                                          // never empty: a whole tile has more than 128 rows
        mfma16_tile<DT_I8, 128, 256, 2, 4, 3, 64, false, false, 16>(g, tc, 0, g.K, nullptr, lds, sc);
}

hipError_t launch_mixed(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr int l0 = mfma16_lds_bytes(256, 256, 2, 64, 16), l1 = mfma16_lds_bytes(128, 256, 3, 64, 16);
    // a wave's tail cut in halves adds at most half a wave of programs
    hipLaunchKernelGGL(scaled_mixed_kernel, dim3(programs + 128), dim3(512), (size_t)(l0 > l1 ? l0 : l1), s, a);
    return hipGetLastError();
}

// Operands of any alignment and K: the same LDS image (rows of 128 bytes,
// chunks placed by swizzle_key), filled through registers by loads that need
// no alignment, two stages ahead.
__device__ __forceinline__ uint4 load_chunk(const int8_t *p)
{
    return __builtin_bit_cast(uint4, load_bytes16(p));
}

template <int BM, int BN>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
void scaled_any_kernel(ScaledArgs a)
{
    extern __shared__ uint4 lds[];
    constexpr int ROWS = BM + BN, PER = ROWS / 64, TM = BM / 2, TN = BN / 4, FM = TM / 16, FN = TN / 16;
    const GroupTile t = scaled_tile<BM>(a);
    if (t.group < 0)
        return;
    const GemmArgs g = scaled_args(a, t.group, t.start, t.rows);
    const int64_t m0 = (int64_t)t.row_tile * BM, n0 = (int64_t)t.col_tile * BN;
    const int64_t last_row = (g.M - m0 < BM ? g.M - m0 : BM) - 1, last_col = (g.N - n0 < BN ? g.N - n0 : BN) - 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave / 4, wn = wave % 4;
    // this thread's chunks: chunk tid % 8 of stage rows tid / 8 + 64 i
    const int chunk = tid % 8;
    const int8_t *src[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t r = tid / 8 + 64 * i;
        src[i] = r < BM ? (const int8_t *)g.A + (m0 + (r < last_row ? r : last_row)) * g.lda
                        : (const int8_t *)g.B + (n0 + (r - BM < last_col ? r - BM : last_col)) * g.ldb;
        src[i] += 16 * chunk;
    }
    auto put = [&](int buffer, const uint4 (&from)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = tid / 8 + 64 * i;
            lds[(buffer * ROWS + r) * 8 + (chunk ^ swizzle_key<8>(r))] = from[i];
        }
    };
    i32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    const int row = lane & 15, key = swizzle_key<8>(row);
    auto multiply = [&](int buffer) {
        const uint4 *as = lds + (buffer * ROWS + wm * TM + row) * 8;
        const uint4 *bs = lds + (buffer * ROWS + BM + wn * TN + row) * 8;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int c = (4 * ks + (lane >> 4)) ^ key;
            i32x4_t fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[i] = __builtin_bit_cast(i32x4_t, as[16 * i * 8 + c]);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j] = __builtin_bit_cast(i32x4_t, bs[16 * j * 8 + c]);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = mfma_16x16x64(fa[i], fb[j], acc[i][j]);
        }
    };
    // Stage 0 is the one that K cuts, if any, so that the others' loads need
    // no mask; from there two stages are under way in registers.  Loads past
    // the last stage repeat it and are not used.
    const int32_t whole = (int32_t)(g.K / 128), cut = g.K % 128 != 0, stages = whole + cut;
    if (g.alpha != 0.0f && stages > 0) {
        uint4 held[2][PER];
        auto fetch = [&](int32_t v, uint4 (&into)[PER]) {
            const int64_t k0 = ((v < stages ? v : stages - 1) - cut) * 128;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                into[i] = load_chunk(src[i] + k0);
        };
        if (cut) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                held[0][i] = __builtin_bit_cast(
                    uint4, load_masked16(src[i] - 16 * chunk, (int64_t)whole * 128 + 16 * chunk, g.K));
        } else {
            fetch(0, held[0]);
        }
        if (whole > 0)
            fetch(1, held[1]);
        put(0, held[0]);
        lds_barrier();
        if (whole > 0) {
            for (int32_t v = 0; v < stages; v += 2) {
                fetch(v + 2, held[0]);
                multiply(0);
                put(1, held[1]);
                lds_barrier();
                if (v + 1 < stages) {
                    fetch(v + 3, held[1]);
                    multiply(1);
                    put(0, held[0]);
                    lds_barrier();
                }
            }
        } else {
            multiply(0);
        }
        lds_barrier();
    }
    const TileCoord tc{0, 0, (int32_t)t.row_tile, (int32_t)t.col_tile};
    const RowColScales sc{row_scales(a, t.start), col_scales(a, t.group), a.scale_type};
    scaled_epilogue<BM, BN, 2, 4, 256>(g, tc, (float *)lds, m0, n0, acc, sc);
}

template <int BM, int BN>
hipError_t launch_any(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr int stages = 2 * (BM + BN) * 128, lds = stages > scaled_epilogue_lds_bytes(BM, BN)
                                                          ? stages : scaled_epilogue_lds_bytes(BM, BN);
    hipLaunchKernelGGL((scaled_any_kernel<BM, BN>), dim3(programs), dim3(512), (size_t)lds, s, a);
    return hipGetLastError();
}

template <int BM, int BN, int NS>
hipError_t launch(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    hipLaunchKernelGGL((scaled_tile_kernel<BM, BN, NS>), dim3(programs), dim3(512),
                       (size_t)mfma16_lds_bytes(BM, BN, NS, 64, 16), s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_scaled_tile(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    switch (variant) {
    case 0: return launch_any<64, 128>(a, programs, s);
    case 1: return launch_any<128, 128>(a, programs, s);
    case 2: return launch<64, 128, 4>(a, programs, s);
    case 3: return launch<128, 128, 4>(a, programs, s);
    case 4: return launch<128, 128, 2>(a, programs, s);
    case 5: return launch_mixed(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
