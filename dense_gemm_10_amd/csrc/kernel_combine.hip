// Rows brought back to their tokens, and the gradients.  Memory bound: every
// row of z is read once, every output written once, no LDS in the forward
// pass.  A sum is one chain of fused multiply-adds in the order of j, a dot
// product one per lane and column of eight, added over the lanes in a fixed
// order: calls repeat bit for bit.
//
// Measured (MI355X, 8192 tokens, 2 rows each, 4096 bf16, kernel times, operands
// the same from call to call): forward 32 us, 202 MB moved, 6.3 TB/s; gradients
// 51 us, 337 MB, 6.6 TB/s.  With new operands in every call the two together
// take 101 us, 5.3 TB/s.
#include "grouped.hpp"
#include "tokens.hpp"

namespace dg {

namespace {

constexpr int CT = 256;

__device__ __forceinline__ float weight(const CombineArgs &a, int64_t t, int32_t j)
{
    return a.w ? load_as_f32(a.w, a.w_type, t * a.ldw + j) : 1.0f;
}

// A wavefront takes 64 x U pieces of eight columns of one token: the pieces
// of KB rows of z are loaded before the first is used.  GRAD: without weights
// the call is a gradient's, whose rows nothing reads again (8192 tokens, 2
// rows, 4096 bf16, with the dispatch: 89 us with plain loads, 78 so; rows with
// weights are read by their gradient, which with them is 107 instead of 101).
template <int TZ, int TY, int KB, int U, bool GRAD>
__global__ __launch_bounds__(CT) void combine_kernel(CombineArgs a)
{
    constexpr int EZ = elem_bytes<TZ>(), EY = elem_bytes<TY>();
    constexpr int SEG = 64 * U * 8;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t segs = (uint32_t)((a.width + SEG - 1) / SEG);
    const int64_t units = a.tokens * segs, step = (int64_t)gridDim.x * (CT / 64);
    for (int64_t unit = (int64_t)blockIdx.x * (CT / 64) + wave; unit < units; unit += step) {
        const int64_t t = unit / segs, first = (unit - t * segs) * SEG;
        float sum[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[u][e] = 0.0f;
        int n[U];                                  // columns of the piece
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t left = a.width - (first + (u * 64 + lane) * 8);
            n[u] = left < 0 ? 0 : left > 8 ? 8 : (int)left;
        }
        for (int32_t j0 = 0; j0 < a.top_k; j0 += KB) {
            Raw8<TZ> v[KB][U];
            bool in[KB];
            float w[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int32_t p = j0 + j < a.top_k ? a.place[t * a.top_k + j0 + j] : -1;
                in[j] = p >= 0 && p < a.limit;
                if (!in[j])
                    continue;
                w[j] = weight(a, t, j0 + j);
                const char *row = a.z + (int64_t)p * a.ldz;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (n[u] > 0)
                        v[j][u] = load_raw8<TZ, GRAD>(row + (first + (u * 64 + lane) * 8) * EZ, n[u]);
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (!in[j])
                    continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum[u][e] = fmaf(w[j], raw_value<TZ>(v[j][u], e), sum[u][e]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (n[u] == 0)
                continue;
            char *dst = a.y + t * a.ldy + (first + (u * 64 + lane) * 8) * EY;
            if (a.beta != 0.0f) {
                const Raw8<TY> old = load_raw8<TY>(dst, n[u]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[u][e] = fmaf(a.beta, raw_value<TY>(old, e), sum[u][e]);
            }
            store_8<TY>(dst, sum[u], n[u]);
        }
    }
}

// Sum over the 64 lanes, in a fixed order; in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        v += __shfl_xor(v, d);
    return v;
}

// NW wavefronts take one token: dy's pieces once for KB rows of z, whose dot
// products with dy are summed over the lanes at the end.
template <int TZ, int TY, int KB, int NW>
__global__ __launch_bounds__(CT) void combine_grad_kernel(CombineArgs a)
{
    constexpr int EZ = elem_bytes<TZ>(), EY = elem_bytes<TY>(), NT = 64 * NW, PER = CT / NT;
    __shared__ float part[CT / 64][KB];
    const int tid = threadIdx.x, sub = tid % NT;
    const int mine = __builtin_amdgcn_readfirstlane(tid / NT);        // token of the workgroup
    const int64_t step = (int64_t)gridDim.x * PER;
    for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + mine;
        const bool live = t < a.tokens;
        for (int32_t j0 = 0; j0 < a.top_k; j0 += KB) {
            float dot[KB], w[KB];
            bool in[KB];
            const char *zr[KB];
            char *dr[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int32_t p = live && j0 + j < a.top_k ? a.place[t * a.top_k + j0 + j] : -1;
                in[j] = p >= 0 && p < a.limit;
                dot[j] = 0.0f;
                w[j] = in[j] && a.dz ? weight(a, t, j0 + j) : 0.0f;
                zr[j] = a.z + (int64_t)(in[j] ? p : 0) * a.ldz;
                dr[j] = a.dz + (int64_t)(in[j] ? p : 0) * a.lddz;
            }
            for (int64_t c = (int64_t)sub * 8; live && c < a.width; c += NT * 8) {
                const int n = a.width - c > 8 ? 8 : (int)(a.width - c);
                const Raw8<TY> g = load_raw8<TY>(a.y + t * a.ldy + c * EY, n);
                Raw8<TZ> v[KB];
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < KB; ++j)
                        if (in[j])
                            v[j] = load_raw8<TZ>(zr[j] + c * EZ, n);
                }
                if (a.dz) {
#pragma unroll
                    for (int j = 0; j < KB; ++j) {
                        if (!in[j])
                            continue;
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = w[j] * raw_value<TY>(g, e);
                        store_8<TZ>(dr[j] + c * EZ, o, n);
                    }
                }
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < KB; ++j) {
                        if (!in[j])
                            continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dot[j] = fmaf(raw_value<TY>(g, e), raw_value<TZ>(v[j], e), dot[j]);
                    }
                }
            }
            if (!a.dw)
                continue;
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float v = wave_sum(dot[j]);
                if ((tid & 63) == 0)
                    part[tid >> 6][j] = v;
            }
            __syncthreads();
            if (live && sub < KB && j0 + sub < a.top_k) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    v += part[mine * NW + i][sub];
                const int64_t at = t * a.top_k + j0 + sub;
                if (a.w_type == DT_F32)
                    ((float *)a.dw)[at] = v;
                else
                    ((uint16_t *)a.dw)[at] = a.w_type == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v);
            }
            __syncthreads();
        }
    }
}

dim3 capped(int64_t workgroups)
{
    return dim3((unsigned)(workgroups < (1 << 20) ? workgroups : 1 << 20));
}

template <int TZ, int TY, int KB, int U>
void combine_launch(const CombineArgs &a, hipStream_t s)
{
    const int64_t units = a.tokens * ((a.width + 64 * U * 8 - 1) / (64 * U * 8));
    const dim3 grid = capped((units + CT / 64 - 1) / (CT / 64));
    if (a.w)
        hipLaunchKernelGGL((combine_kernel<TZ, TY, KB, U, false>), grid, dim3(CT), 0, s, a);
    else
        hipLaunchKernelGGL((combine_kernel<TZ, TY, KB, U, true>), grid, dim3(CT), 0, s, a);
}

// KB: the rows of a token, up to eight at once.
template <int TZ, int TY>
void combine_choice(const CombineArgs &a, hipStream_t s)
{
    if (a.top_k <= 1)
        combine_launch<TZ, TY, 1, 2>(a, s);
    else if (a.top_k == 2)
        combine_launch<TZ, TY, 2, 1>(a, s);
    else if (a.top_k <= 4)
        combine_launch<TZ, TY, 4, 1>(a, s);
    else
        combine_launch<TZ, TY, 8, 2>(a, s);
}

template <int TZ, int TY, int KB>
void grad_launch(const CombineArgs &a, hipStream_t s)
{
    if (a.width <= 1024)
        hipLaunchKernelGGL((combine_grad_kernel<TZ, TY, KB, 1>), capped((a.tokens + 3) / 4), dim3(CT), 0, s, a);
    else
        hipLaunchKernelGGL((combine_grad_kernel<TZ, TY, KB, 4>), capped(a.tokens), dim3(CT), 0, s, a);
}

template <int TZ, int TY>
void grad_choice(const CombineArgs &a, hipStream_t s)
{
    if (a.top_k <= 1)
        grad_launch<TZ, TY, 1>(a, s);
    else if (a.top_k == 2)
        grad_launch<TZ, TY, 2>(a, s);
    else if (a.top_k <= 4)
        grad_launch<TZ, TY, 4>(a, s);
    else
        grad_launch<TZ, TY, 8>(a, s);
}

} // namespace

hipError_t launch_combine(const CombineArgs &a, hipStream_t s)
{
    if (a.z_type == DT_F32)
        combine_choice<DT_F32, DT_F32>(a, s);
    else if (a.z_type == DT_BF16)
        a.y_type == DT_F32 ? combine_choice<DT_BF16, DT_F32>(a, s) : combine_choice<DT_BF16, DT_BF16>(a, s);
    else
        a.y_type == DT_F32 ? combine_choice<DT_F16, DT_F32>(a, s) : combine_choice<DT_F16, DT_F16>(a, s);
    return hipGetLastError();
}

hipError_t launch_combine_grad(const CombineArgs &a, hipStream_t s)
{
    if (a.z_type == DT_F32)
        grad_choice<DT_F32, DT_F32>(a, s);
    else if (a.z_type == DT_BF16)
        a.y_type == DT_F32 ? grad_choice<DT_BF16, DT_F32>(a, s) : grad_choice<DT_BF16, DT_BF16>(a, s);
    else
        a.y_type == DT_F32 ? grad_choice<DT_F16, DT_F32>(a, s) : grad_choice<DT_F16, DT_F16>(a, s);
    return hipGetLastError();
}

} // namespace dg
