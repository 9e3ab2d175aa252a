// Products with 4-bit weights (stream.hpp): W's codes go from memory into
// registers 16 bytes per lane, become MFMA operands by two instructions per
// pair of weights, and the scales multiply fp32 sums.
//
// Codes to operands.  A 16-bit float with exponent 4 and the code q in its
// top four fraction bits is 16 + q, exactly: bf16 0x4180 | q << 3, fp16
// 0x4c00 | q << 6.  One shift and one and-or of a word of eight codes give
// codes j and j + 4 as the two halves of a register, so the operand's
// k-order is 0 4 1 5 2 6 3 7; A is staged in LDS in the same order.  With U
// = sum a (16 + q) and S = sum a over the k of one scale, both in fp32,
//   sum a scale (q - zero) = scale (U - (16 + zero) S).
// S comes from one more MFMA per step, against a column of ones, where a
// wavefront has one column block and the matrix pipe is idle anyway, and is
// formed as A is staged, once per workgroup, where it has more.
// Nothing is rounded to 16 bits; the subtraction costs the sums at most
// five bits of fp32 (|16 + q| <= 31 against |q - zero| of a few units), and an
// output whose sums are not finite is formed again (defined_product).
//
// Measured (MI355X): one row through 16384 x 8192 (fp16, groups of 64) 17.4
// us, 4.2 TB/s, bound by the codes' bytes; through 4096 x 4096 5.1 us in a
// replayed graph, 7.4 us called from the host, bound by launch and latency;
// 2048 rows through 4096 x 4096 (bf16, groups of 128) 84-86 us, 0.8 PFLOP/s,
// bound by the panel's chain of stage, barrier and first operand reads, which
// two wavefronts per SIMD do not cover.
//
// Work split.  A workgroup is NW x KW wavefronts and owns 16 FM rows x 16
// FN NW columns; it walks K in panels of 128 KW TS.  Per panel the
// workgroup stages A's rows (MR <= 16 FM at most) and the panel's scales in LDS, and wavefront
// (n, w) takes its 16 FN columns over the steps w, w + KW, ... of 128 k.
// The next panel's codes, A and scales are loaded into registers before
// this panel is multiplied, so memory is never waited for in the loop.
// A through LDS and not straight into registers: there each wavefront's A
// pieces take four times the load instructions of its codes, and the
// vector-memory path, not HBM, bounds the kernel (16384 x 8192, one row: 31
// us; 16 rows: 46 us).
//
// Codes to MFMA steps.  Lane 16 g + c loads codes 32 g .. 32 g + 31 of row
// c, 64 bytes of each row, and a 4 x 4 exchange between the four 16-lane
// groups (two half-wave swaps, two quarter swaps) gives register t of group
// g the codes 32 t + 8 g .. + 7: MFMA t of the step then covers 32
// consecutive k, which share a scale for any group size that is a multiple
// of 32.  SPG: MFMA steps that surely share a scale (1, 2 or 4: group sizes
// that are multiples of 32, 64 or 128).
#pragma once
#include "stream.hpp"
#include <type_traits>

namespace dg {

namespace {

constexpr int QK = 128;            // k of one step of a wavefront

// Exchange between the two registers: lanes 32-63 of x with lanes 0-31 of y.
__device__ __forceinline__ void swap_halves(uint32_t &x, uint32_t &y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}
// Lanes 16-31 of x with lanes 0-15 of y, and 48-63 of x with 32-47 of y.
__device__ __forceinline__ void swap_quarters(uint32_t &x, uint32_t &y)
{
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}

// w[t] of lane group g becomes w[g] of lane group t.
__device__ __forceinline__ void transpose_groups(uint32_t (&w)[4])
{
    swap_halves(w[0], w[2]);
    swap_halves(w[1], w[3]);
    swap_quarters(w[0], w[1]);
    swap_quarters(w[2], w[3]);
}

// 16.0 in both halves of a register, opaque to the compiler: an and-or takes
// its mask and one more constant only if one of them is in a vector register.
template <int T>
__device__ __forceinline__ uint32_t sixteen()
{
    uint32_t v = T == DT_F16 ? 0x4c004c00u : 0x41804180u;
    asm("" : "+v"(v));
    return v;
}

// Eight codes of a word as an operand of values 16 + q, in k-order 0 4 1 5
// 2 6 3 7.
template <int T>
__device__ __forceinline__ uint4 codes_to_operand(uint32_t w, uint32_t base)
{
    constexpr uint32_t mask = T == DT_F16 ? 0x03c003c0u : 0x00780078u;
    if constexpr (T == DT_F16)
        return make_uint4((w << 6 & mask) | base, (w << 2 & mask) | base, (w >> 2 & mask) | base,
                          (w >> 6 & mask) | base);
    else
        return make_uint4((w << 3 & mask) | base, (w >> 1 & mask) | base, (w >> 5 & mask) | base,
                          (w >> 9 & mask) | base);
}

// Eight consecutive 16-bit values of A in the same order.
__device__ __forceinline__ uint4 reorder_a(uint4 v)
{
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u),
                      __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

// Sum of a piece's eight values: four dot products with (1, 1) in fp32.
template <int T>
__device__ __forceinline__ float sum_of_piece(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == DT_F16) {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            s = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w[i]),
                                       f16x2{(_Float16)1.0f, (_Float16)1.0f}, s, false);
        } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[i]),
                                                bf16x2{(__bf16)1.0f, (__bf16)1.0f}, s, false);
        }
    }
    return s;
}

// Sum over aligned runs of 4, 8 or 16 lanes, in every lane of the run
// (exchanges inside quads, then mirrored halves of 8, then of 16 lanes).
template <int LANES>
__device__ __forceinline__ float run_sum(float v)
{
    auto add = [&](auto ctrl) {
        v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
            0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    add(std::integral_constant<int, 0xb1>{});          // lane ^ 1
    add(std::integral_constant<int, 0x4e>{});          // lane ^ 2
    if (LANES >= 8)
        add(std::integral_constant<int, 0x141>{});     // 7 - lane in 8 lanes
    if (LANES >= 16)
        add(std::integral_constant<int, 0x140>{});     // 15 - lane in 16 lanes
    return v;
}

// One output from the definition, k by k in fp32, in the order of the kernel
// that takes every operand: where U or S is not finite (an infinity in A, or
// values whose 31-fold sum passes fp32), U - (16 + zero) S does not give what
// the formula does.  x: the row of A; q, scales, zeros (null: 8): the
// column's, from its first code.  K is a multiple of 32.  One thread per
// output: 2048 rows of NaN through 4096 x 4096 take 135 us instead of 84, of
// infinities that meet no weight of zero 59 ms.  Not inlined: in line it
// changed the K loop's instructions (one token through 16384 x 8192: 18.0 us;
// called 17.5, without it 17.4).  What the test for it costs: nothing to 1.5 %
// (2048 rows of 4096 x 4096: 83.1 -> 84.3 us).
template <int T>
__device__ __noinline__ float defined_product(const uint16_t *x, const uint8_t *q, const void *scales,
                                              const uint8_t *zeros, int32_t scale_type, uint32_t K,
                                              uint32_t per_scale)
{
    float sum = 0.0f;
#pragma unroll 1
    for (uint32_t k = 0; k < K && sum == sum; k += 2) {        // NaN stays NaN
        const uint32_t j = k / per_scale;
        const float scale = load_as_f32(scales, scale_type, j);
        const int32_t zero = zeros ? zeros[j] & 15 : 8, two = q[k / 2];
        sum = fmaf(half_to_f32<T>(x[k]), (float)((two & 15) - zero) * scale, sum);
        sum = fmaf(half_to_f32<T>(x[k + 1]), (float)((two >> 4) - zero) * scale, sum);
    }
    return sum;
}

// LDS of a workgroup: A's panel, rows 16 bytes apart in banks, the panel's
// (scale, -(16 + zero)) pairs and the sums of A over each scale's k; or the
// wavefronts' sums at the end.
template <int SPG, int FM, int FN, int NW, int KW, int TS, int MR>
struct QPanel {
    static constexpr int K = QK * KW * TS;            // k of a panel
    static constexpr int E = K / (32 * SPG);          // scales of a row
    static constexpr int COLS = 16 * FN * NW;
    static constexpr int NT = 64 * NW * KW;
    static constexpr int A_LD = K + 8;                // 16-bit elements
    static constexpr int S_LD = E + 1;                // float pairs
    static constexpr int A_BYTES = MR * A_LD * 2;
    static constexpr int A_PER = MR * K / 8 / NT;         // 16-byte pieces of A per thread
    static constexpr int S_ALL = COLS * E;                // scales of the panel
    static constexpr int S_PER = (S_ALL + NT - 1) / NT;   // ... per thread
    static constexpr int PIECES = A_PER + S_PER;          // loads of a thread for a panel
    static constexpr int SUM_LD = COLS + 4;
    static constexpr int SUM_AT = (A_BYTES + COLS * S_LD * 8 + 15) / 16 * 16;   // sums[E][16 FM]
    static constexpr bool STAGED_SUMS = FN > 1;
    static constexpr int PANEL = (SUM_AT + (STAGED_SUMS ? E * 16 * FM * 4 : 0) + 15) / 16 * 16;
    // Two panels in LDS, with one barrier each, where a wavefront has four
    // blocks or more (128 rows of 8192 x 8192 on 32 x 128: 40 us, with one
    // panel 43); smaller ones live from many workgroups per CU, which two
    // panels halve (512 rows of 4096 x 4096 on 32 x 32: 74 us against 55).
    static constexpr bool TWO = FM * FN >= 4;
    static constexpr int LOOP = TWO ? 2 * PANEL : PANEL;
    static constexpr int STORE = KW * 16 * FM * SUM_LD * 4;
    static constexpr int BYTES = LOOP > STORE ? LOOP : STORE;
    static_assert(A_PER * NT * 8 == MR * K, "A split");
};

template <int T, bool S32, bool ZEROS, int SPG, int FM, int FN, int NW, int KW, int TS, int MR>
__global__ __launch_bounds__(64 * NW * KW)
__attribute__((amdgpu_waves_per_eu(FM * FN >= 32 ? 1 : FM * FN >= 8 ? 2 : 4)))
void qweight_stream_kernel(QweightArgs a, FastDiv by_group)
{
    using frag_t = typename frag_of<T>::type;
    using P = QPanel<SPG, FM, FN, NW, KW, TS, MR>;
    extern __shared__ uint4 lds[];
    GroupTile t;
    constexpr int G = 8;
    if (a.offsets) {
        t = find_group_tile<16 * FM, G>(a.offsets, a.groups, a.rows, a.tiles_n, blockIdx.x);
        if (t.group < 0)
            return;
    } else {
        // the same order without groups: contiguous runs to the XCDs, bands
        // of G row tiles walked column by column, so that an XCD's running
        // tiles share codes and rows of A
        const uint32_t tm = ((uint32_t)a.rows + 16 * FM - 1) / (16 * FM);
        const uint32_t N = tm * a.tiles_n, x = blockIdx.x % kNumXcd, r = N % kNumXcd;
        const uint32_t L = x * (N / kNumXcd) + (x < r ? x : r) + blockIdx.x / kNumXcd;
        const uint32_t band = L / (G * a.tiles_n), o = L - band * (G * a.tiles_n);
        const uint32_t left = tm - band * G, h = left < G ? left : G;
        t = GroupTile{0, 0, a.rows, band * G + o % h, o / h};
    }
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nw = wave % NW, kw = wave / NW;
    const int64_t m0 = (int64_t)t.row_tile * (16 * FM), n0 = (int64_t)t.col_tile * P::COLS;
    const int rows = (int)(t.rows - m0 < 16 * FM ? t.rows - m0 : 16 * FM);
    const int cols = (int)(a.N - n0 < P::COLS ? a.N - n0 : P::COLS);

    // Each operand: a uniform base and a 32-bit byte offset per lane
    // (checked on the host to fit).  Columns past the last repeat it.
    const global_base ab = uniform_base((const uint16_t *)a.A + (t.start + m0) * a.lda);
    const global_base qb = uniform_base(a.Q + t.group * a.stride_q + n0 * a.ldq);
    const int64_t s0 = t.group * a.stride_s + n0 * a.lds;
    const global_base sb = uniform_base((const char *)a.scales + s0 * (S32 ? 4 : 2));
    const global_base zb = uniform_base(a.zeros + (ZEROS ? s0 : 0));
    const uint32_t K = (uint32_t)a.K;      // a multiple of 32 below 2^31 (checked on the host)
    uint32_t qo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const uint32_t n = 16 * (FN * nw + j) + c;
        qo[j] = (n < (uint32_t)cols ? n : cols - 1) * (uint32_t)a.ldq;
    }
    // panel buffer b
    auto a_lds = [&](int b) { return (uint16_t *)((char *)lds + b * P::PANEL); };
    auto s_lds = [&](int b) { return (float2 *)((char *)lds + b * P::PANEL + P::A_BYTES); };
    auto sum_lds = [&](int b) { return (float *)((char *)lds + b * P::PANEL + P::SUM_AT); };

    struct Codes {
        uint4 q[TS][FN];
    };
    struct Staged {
        uint4 a[P::A_PER];
        // as loaded: widened here, they would have to arrive first
        std::conditional_t<S32, uint32_t, uint16_t> s[P::S_PER];
        uint8_t z[P::S_PER];
    };
    // k past K reads the row's last codes: A is zero there.
    auto load_code = [&](Codes &r, uint32_t k0, int i, int j) {
        const uint32_t k = k0 + (kw + i * KW) * QK + 32 * kg;
        r.q[i][j] = load16_at(qb, qo[j] + (k < K ? k : K - 32) / 2);
    };
    auto load_codes = [&](Codes &r, uint32_t k0) {
#pragma unroll
        for (int i = 0; i < TS; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                load_code(r, k0, i, j);
    };
    // one piece per thread of the panel: 0 .. A_PER - 1 of A, then of the scales
    auto load_piece = [&](Staged &r, uint32_t k0, int p) {
        if (p < P::A_PER) {
            const int piece = tid + p * P::NT, row = piece / (P::K / 8);
            const uint32_t k = k0 + piece % (P::K / 8) * 8;
            // few rows: no load for those that are not there; many: the last
            // row again, without a branch
            if (P::TWO || (row < rows && k < K))
                r.a[p] = load16_at(ab, (uint32_t)(row < rows ? row : rows - 1) * (uint32_t)(2 * a.lda) +
                                           2 * (k < K ? k : 0));
        } else {
            const int i = p - P::A_PER;
            const int all = tid + i * P::NT, e = all < P::S_ALL ? all : P::S_ALL - 1;
            const int n = e / P::E;
            const uint32_t k = k0 + e % P::E * (32 * SPG);
            const uint32_t at = (uint32_t)(n < cols ? n : cols - 1) * (uint32_t)a.lds +
                                fastdiv(k < K ? k : K - 1, by_group);
            if constexpr (S32)
                r.s[i] = load_at<uint32_t>(sb, at * 4);
            else
                r.s[i] = load_at<uint16_t>(sb, at * 2);
            if (ZEROS)
                r.z[i] = load_at<uint8_t>(zb, at);
        }
    };
    auto load_panel = [&](Staged &r, uint32_t k0) {
#pragma unroll
        for (int p = 0; p < P::PIECES; ++p)
            load_piece(r, k0, p);
    };
    const bool f16_scale = a.scale_type == DT_F16;
    auto store_piece = [&](const Staged &r, uint32_t k0, int b, int p) {
        if (p < P::A_PER) {
            const int piece = tid + p * P::NT, row = piece / (P::K / 8), at = piece % (P::K / 8) * 8;
            // one scale's pieces are 4 SPG consecutive lanes of one row
            const uint4 v = k0 + at < K ? r.a[p] : make_uint4(0u, 0u, 0u, 0u);
            float sum = 0.0f;
            if constexpr (P::STAGED_SUMS)
                sum = run_sum<4 * SPG>(sum_of_piece<T>(v));
            if (P::TWO || row < rows) {
                *(uint4 *)(a_lds(b) + row * P::A_LD + at) = reorder_a(v);
                if (P::STAGED_SUMS && piece % (4 * SPG) == 0)
                    sum_lds(b)[at / (32 * SPG) * (16 * FM) + row] = sum;
            }
        } else {
            const int i = p - P::A_PER, e = tid + i * P::NT;
            float f;
            if constexpr (S32)
                f = __uint_as_float(r.s[i]);
            else
                f = f16_scale ? f16_to_f32(r.s[i]) : bf16_to_f32(r.s[i]);
            const float h = ZEROS ? -16.0f - (float)(r.z[i] & 15) : -24.0f;
            // past K a scale of zero: the sums there are zero, whatever the scale
            const bool in = k0 + e % P::E * (32 * SPG) < K;
            if (e < P::S_ALL)
                s_lds(b)[e / P::E * P::S_LD + e % P::E] = make_float2(in ? f : 0.0f, h);
        }
    };
    auto store_panel = [&](const Staged &r, uint32_t k0, int b) {
#pragma unroll
        for (int p = 0; p < P::PIECES; ++p)
            store_piece(r, k0, b, p);
    };

    const f32x4_t none{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t base = sixteen<T>();
    const uint32_t one2 = T == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
    const frag_t ones = __builtin_bit_cast(frag_t, make_uint4(one2, one2, one2, one2));
    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = none;
    int a_at[FM];                          // rows past the last repeat it
#pragma unroll
    for (int i = 0; i < FM; ++i)
        a_at[i] = (16 * i + c < rows ? 16 * i + c : rows - 1) * P::A_LD + 8 * kg;
    const int s_at = (16 * FN * nw + c) * P::S_LD;

    // `between(slot)` is called after each column block's MFMAs, slots 0 ..
    // SLOTS - 1 of a panel
    constexpr int SLOTS = TS * 4 * FN;
    auto multiply = [&](const Codes &r, int b, uint32_t k0, auto &&between) {
        const uint16_t *a_buf = a_lds(b);
        const float2 *s_row = s_lds(b) + s_at;
        const float *sums = sum_lds(b) + 4 * kg;
#pragma unroll
        for (int i = 0; i < TS; ++i) {
            const int step = kw + i * KW;          // of the panel
            if (k0 + step * QK >= K)
                break;
            sched_fence();                         // one step's operands in registers at a time
            uint32_t w[FN][4];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                w[j][0] = r.q[i][j].x;
                w[j][1] = r.q[i][j].y;
                w[j][2] = r.q[i][j].z;
                w[j][3] = r.q[i][j].w;
                transpose_groups(w[j]);
            }
            f32x4_t u[FM][FN], sum[FM];
            float2 sc[FN];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const bool first = m % SPG == 0;
                const int e = step * (4 / SPG) + m / SPG;
                if (first) {               // read early: the MFMAs cover the latency
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        sc[j] = s_row[j * 16 * P::S_LD + e];
                    if constexpr (P::STAGED_SUMS)
#pragma unroll
                        for (int x = 0; x < FM; ++x)
                            sum[x] = *(const f32x4_t *)(sums + e * (16 * FM) + 16 * x);
                }
                frag_t af[FM];
#pragma unroll
                for (int x = 0; x < FM; ++x) {
                    af[x] = *(const frag_t *)(a_buf + a_at[x] + step * QK + 32 * m);
                    if constexpr (!P::STAGED_SUMS)
                        sum[x] = mfma_16x16x32(af[x], ones, first ? none : sum[x]);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const frag_t b = __builtin_bit_cast(frag_t, codes_to_operand<T>(w[j][m], base));
#pragma unroll
                    for (int x = 0; x < FM; ++x)
                        u[x][j] = mfma_16x16x32(af[x], b, first ? none : u[x][j]);
                    between((4 * i + m) * FN + j);
                }
                if (m % SPG == SPG - 1) {
                    sched_fence();
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const float2 s = sc[j];
#pragma unroll
                        for (int x = 0; x < FM; ++x)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[x][j][v] = fmaf(s.x, fmaf(s.y, sum[x][v], u[x][j][v]), acc[x][j][v]);
                        // finished here: otherwise the compiler puts these additions off past
                        // the barrier and keeps every u and sum until then
#pragma unroll
                        for (int x = 0; x < FM; ++x)
                            asm volatile("" : "+v"(acc[x][j]));
                    }
                }
            }
        }
    };

    if (a.alpha != 0.0f && K > 0) {
        Codes now, next;
        Staged panel;
        load_codes(now, 0);
        load_panel(panel, 0);
        store_panel(panel, 0, 0);
        if constexpr (P::TWO) {
            // the panel after the next is on its way (past K: a harmless
            // repeat) while this one is multiplied and the next one staged
            load_panel(panel, P::K);
            lds_barrier();
            int b = 0;
            for (uint32_t k0 = 0;; b ^= 1) {
                const uint32_t k1 = k0 + P::K;
                if (k1 >= K) {
                    multiply(now, b, k0, [](int) {});
                    break;
                }
                // The next panel's codes, the staging of its rows and scales
                // and the loads of the panel after it, one at a time between
                // the MFMAs: in one block before them they keep the matrix
                // pipe waiting for the issue of the 8 wavefronts' loads (2048
                // rows of 4096 x 4096: 98 us, in one block 104).
                multiply(now, b, k0, [&](int slot) {
                    constexpr int JOBS = TS * FN + P::PIECES;
#pragma unroll
                    for (int job = 0; job < JOBS; ++job) {
                        if (job * SLOTS / JOBS != slot)
                            continue;
                        if (job < TS * FN) {
                            load_code(next, k1, job / FN, job % FN);
                        } else {
                            store_piece(panel, k1, b ^ 1, job - TS * FN);
                            load_piece(panel, k1 + P::K, job - TS * FN);
                        }
                    }
                });
                lds_barrier();
                now = next;
                k0 = k1;
            }
        } else {
            lds_barrier();
            for (uint32_t k0 = 0;;) {
                const uint32_t k1 = k0 + P::K;
                if (k1 >= K) {
                    multiply(now, 0, k0, [](int) {});
                    break;
                }
                load_panel(panel, k1);
                load_codes(next, k1);
                multiply(now, 0, k0, [](int) {});
                lds_barrier();             // every wavefront is done with this panel
                store_panel(panel, k1, 0);
                lds_barrier();
                now = next;
                k0 = k1;
            }
        }
        lds_barrier();
    }

    // the KW wavefronts' sums, added in wavefront order, and the epilogue
    GemmArgs g{};
    g.M = t.rows;
    g.N = a.N;
    g.ldc = a.ldc;
    g.alpha = a.alpha;
    g.beta = a.beta;
    g.act = a.act;
    g.c_type = a.c_type;
    g.bias_type = a.bias_type;
    g.C = (char *)a.C + (int64_t)t.start * a.ldc * (a.c_type == DT_F32 ? 4 : 2);
    g.bias = a.bias ? (const char *)a.bias + t.group * a.stride_bias * (a.bias_type == DT_F32 ? 4 : 2)
                    : nullptr;
    float *part = (float *)lds;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                part[(kw * 16 * FM + 16 * i + 4 * kg + v) * P::SUM_LD + 16 * (FN * nw + j) + c] =
                    acc[i][j][v];
    lds_barrier();
    auto from_definition = [&](int r, int n) {
        const int64_t s_at = s0 + n * a.lds;
        return defined_product<T>((const uint16_t *)a.A + (t.start + m0 + r) * a.lda,
                                  a.Q + t.group * a.stride_q + (n0 + n) * a.ldq,
                                  (const char *)a.scales + s_at * (S32 ? 4 : 2), ZEROS ? a.zeros + s_at : nullptr,
                                  a.scale_type, K, (uint32_t)(a.group_size < a.K ? a.group_size : a.K));
    };
    // Large tiles: four columns per thread, one store each, where C's rows
    // allow it (2048 rows of 4096 x 4096: 85 us, one by one 98).
    constexpr int RUN = 16 * FM * P::COLS >= 8 * P::NT ? 4 : 1;
    const int cs = a.c_type == DT_F32 ? 4 : 2;
    const bool whole = RUN > 1 && a.ldc % RUN == 0 && (uintptr_t)g.C % (RUN * cs) == 0;
    for (int o = tid; o < 16 * FM * P::COLS / RUN; o += P::NT) {
        const int r = o / (P::COLS / RUN), n = o % (P::COLS / RUN) * RUN;
        if (r >= rows || n >= cols)
            continue;
        float v[RUN];
#pragma unroll
        for (int e = 0; e < RUN; ++e) {
            v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w)
                v[e] += part[(w * 16 * FM + r) * P::SUM_LD + n + e];
        }
        float all = v[0];                      // not finite if one of the run is not
#pragma unroll
        for (int e = 1; e < RUN; ++e)
            all += v[e];
        if (__builtin_expect(!(fabsf(all) < INFINITY), 0)) {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (n + e < cols && !(fabsf(v[e]) < INFINITY))
                    v[e] = from_definition(r, n + e);
        }
        if constexpr (RUN > 1) {
            if (whole && n + RUN <= cols) {
                float bias[RUN];
#pragma unroll
                for (int e = 0; e < RUN; ++e)
                    bias[e] = g.bias ? load_as_f32(g.bias, g.bias_type, n0 + n + e) : 0.0f;
                run_epilogue<RUN>(g, 0, m0 + r, n0 + n, g.N, false, v, bias);
                char *dst = (char *)g.C + ((m0 + r) * g.ldc + n0 + n) * cs;
                if (g.c_type == DT_F32) {
                    store16(dst, v[0], v[1], v[2], v[3]);
                } else {
                    uint32_t h[RUN];
#pragma unroll
                    for (int e = 0; e < RUN; ++e)
                        h[e] = g.c_type == DT_F16 ? f32_to_f16(v[e]) : f32_to_bf16(v[e]);
                    *(uint2 *)dst = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                }
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < RUN; ++e)
            if (n + e < cols)
                store_c(g, 0, m0 + r, n0 + n + e, epilogue_value(g, 0, m0 + r, n0 + n + e, v[e]));
    }
}

template <int T, bool S32, bool ZEROS, int SPG, int FM, int FN, int NW, int KW, int TS, int MR>
hipError_t launch(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    hipLaunchKernelGGL((qweight_stream_kernel<T, S32, ZEROS, SPG, FM, FN, NW, KW, TS, MR>),
                       dim3(programs), dim3(64 * NW * KW), (QPanel<SPG, FM, FN, NW, KW, TS, MR>::BYTES),
                       s, a, fastdiv_make((uint32_t)(a.group_size < a.K ? a.group_size : a.K)));
    return hipGetLastError();
}

template <bool S32, bool ZEROS, int SPG, int... SHAPE>
hipError_t launch_typed(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    return a.a_type == DT_F16 ? launch<DT_F16, S32, ZEROS, SPG, SHAPE...>(a, programs, s)
                              : launch<DT_BF16, S32, ZEROS, SPG, SHAPE...>(a, programs, s);
}

template <int SPG, int... SHAPE>
hipError_t launch_scaled(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    if (a.scale_type == DT_F32)
        return a.zeros ? launch_typed<true, true, SPG, SHAPE...>(a, programs, s)
                       : launch_typed<true, false, SPG, SHAPE...>(a, programs, s);
    return a.zeros ? launch_typed<false, true, SPG, SHAPE...>(a, programs, s)
                   : launch_typed<false, false, SPG, SHAPE...>(a, programs, s);
}

// SHAPE: FM, FN, NW, KW, TS, MR
template <int... SHAPE>
hipError_t launch_shape(const QweightArgs &a, uint32_t programs, hipStream_t s)
{
    if (a.group_size % 128 == 0)
        return launch_scaled<4, SHAPE...>(a, programs, s);
    if (a.group_size % 64 == 0)
        return launch_scaled<2, SHAPE...>(a, programs, s);
    return launch_scaled<1, SHAPE...>(a, programs, s);
}

} // namespace

} // namespace dg
