// 8-bit products with few rows per group, and of operands of any alignment.
//
// As in stream.hpp, a workgroup owns 16 FM rows x 16 FN columns and its KW
// wavefronts take the steps of 128 k in turn; A and B go from memory into
// MFMA operand registers, 16 bytes of a row per lane, by loads that need no
// alignment.  K's last part is masked in A, whose zeros make B's bytes there
// count for nothing.  The wavefronts' integer sums meet in LDS, are added,
// and take scales and epilogue once.
#include "scaled.hpp"
#include "stream.hpp"

namespace dg {

namespace {

__device__ __forceinline__ i32x4_t load_piece(const int8_t *p)
{
    return __builtin_bit_cast(i32x4_t, load_bytes16(p));
}

__device__ __forceinline__ i32x4_t load_piece_masked(const int8_t *row, int64_t k, int64_t K)
{
    return __builtin_bit_cast(i32x4_t, load_masked16(row, k, K));
}

template <int FM, int FN, int KW, int D>
__global__ __launch_bounds__(64 * KW) void scaled_stream_kernel(ScaledArgs a)
{
    constexpr int SK = 128, NT = 64 * KW, TILE = 16 * FM * 16 * FN, LD = 16 * FN + 4;
    extern __shared__ int32_t sums[];
    const GroupTile t = scaled_tile<16 * FM, 16>(a);
    if (t.group < 0)
        return;
    const GemmArgs g = scaled_args(a, t.group, t.start, t.rows);
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)t.row_tile * (16 * FM), n0 = (int64_t)t.col_tile * (16 * FN);
    const int rows = (int)(g.M - m0 < 16 * FM ? g.M - m0 : 16 * FM);
    const int cols = (int)(g.N - n0 < 16 * FN ? g.N - n0 : 16 * FN);

    const int8_t *ap[FM], *bp[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        ap[i] = (const int8_t *)g.A + (m0 + (16 * i + c < rows ? 16 * i + c : rows - 1)) * g.lda;
#pragma unroll
    for (int j = 0; j < FN; ++j)
        bp[j] = (const int8_t *)g.B + (n0 + (16 * j + c < cols ? 16 * j + c : cols - 1)) * g.ldb;

    struct Step {
        i32x4_t a[2][FM], b[2][FN];
    };
    auto load = [&](Step &s, int64_t k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                s.b[h][j] = load_piece(bp[j] + k + 64 * h + 16 * kg);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                s.a[h][i] = load_piece(ap[i] + k + 64 * h + 16 * kg);
        }
    };
    i32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = i32x4_t{0, 0, 0, 0};
    auto multiply = [&](const Step &s) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    acc[i][j] = mfma_16x16x64(s.a[h][i], s.b[h][j], acc[i][j]);
    };

    if (g.alpha != 0.0f) {
        // A ring of D steps in registers, whose loads are under way while the
        // step before is multiplied.  Loads past the last whole step repeat it
        // and are not used: with none left out, the compiler can count them.
        // D = 2 only where few wavefronts fit a compute unit anyway: more
        // registers cost wavefronts (13 rows, 16384 x 8192, 16 x 64: 30 us
        // with two, 28.3 with one).
        const int32_t full = (int32_t)(g.K / SK);
        int32_t s = wave;
        if (s < full) {
            Step ring[D];
            // Workgroups begin at different steps, so that those running at one
            // time do not all read the same few k of rows a power of two
            // apart (13 rows, 16384 x 8192: 28.3 us without, 26.4 with; 64
            // rows, 4 groups, 4096 x 4096 18.9 and 17.2).
            const int32_t turn = (int32_t)(t.col_tile * 5 % (uint32_t)full);
            auto fetch = [&](Step &r, int32_t at) {
                at = (at < full ? at : full - 1) + turn;
                load(r, (int64_t)(at < full ? at : at - full) * SK);
            };
#pragma unroll
            for (int i = 0; i < D; ++i)
                fetch(ring[i], s + i * KW);
            for (; s + D * KW < full; s += D * KW) {
#pragma unroll
                for (int i = 0; i < D; ++i) {
                    multiply(ring[i]);
                    fetch(ring[i], s + (D + i) * KW);
                }
            }
#pragma unroll
            for (int i = 0; i < D; ++i)
                if (s + i * KW < full)
                    multiply(ring[i]);
        }
        // at most one step is left, the turn of wavefront full mod KW
        const int64_t k0 = (int64_t)full * SK;
        if (k0 < g.K && wave == full % KW) {
            Step last;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + 64 * h + 16 * kg;
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    last.b[h][j] = load_piece_masked(bp[j], k, g.K);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    last.a[h][i] = load_piece_masked(ap[i], k, g.K);
            }
            multiply(last);
        }
    }

    int32_t *mine = sums + wave * (16 * FM * LD);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                mine[(16 * i + 4 * kg + v) * LD + 16 * j + c] = acc[i][j][v];
    lds_barrier();
    const float *sa = row_scales(a, t.start);
    const void *sb = col_scales(a, t.group);
    for (int o = tid; o < TILE; o += NT) {
        const int r = o / (16 * FN), col = o % (16 * FN);
        if (r >= rows || col >= cols)
            continue;
        int32_t sum = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w)
            sum += sums[w * (16 * FM * LD) + r * LD + col];
        const float v =
            (float)sum * (sa ? sa[m0 + r] : 1.0f) * (sb ? load_as_f32(sb, a.scale_type, n0 + col) : 1.0f);
        store_c(g, 0, m0 + r, n0 + col, epilogue_value(g, 0, m0 + r, n0 + col, v));
    }
}

template <int FM, int FN, int KW, int D>
hipError_t launch(const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    constexpr size_t lds = (size_t)KW * 16 * FM * (16 * FN + 4) * 4;
    hipLaunchKernelGGL((scaled_stream_kernel<FM, FN, KW, D>), dim3(programs), dim3(64 * KW), lds, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_scaled_stream(int32_t variant, const ScaledArgs &a, uint32_t programs, hipStream_t s)
{
    switch (variant) {
    case 0: return launch<1, 1, 8, 2>(a, programs, s);
    case 1: return launch<1, 2, 8, 1>(a, programs, s);
    case 2: return launch<1, 2, 4, 2>(a, programs, s);
    case 3: return launch<1, 4, 8, 1>(a, programs, s);
    case 4: return launch<2, 2, 8, 1>(a, programs, s);
    case 5: return launch<2, 4, 8, 1>(a, programs, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace dg
