// Slots sorted by group (a stable counting sort) and rows spread to their
// places.
//
// offsets[e] counts the slots of lower groups; the place of slot s of group
// e is offsets[e] plus the earlier slots of e.  Nothing but counts, so no
// atomic's order can change a result.
//
// Measured (MI355X, kernel times, operands the same from call to call): 16384
// slots on 16 groups 11.8 us of sort_kernel, which reads and writes under 2 MB
// and is bound by latency; then their rows of 4096 bf16 30 us, 202 MB moved,
// 6.7 TB/s; 32 slots with rows of 2048 bf16 in one launch 3.1 us.
#include "grouped.hpp"
#include "tokens.hpp"

namespace dg {

namespace {

// Group of slot s; `groups` for none.
template <typename I>
__device__ __forceinline__ int32_t slot_group(const DispatchArgs &a, uint32_t s)
{
    int64_t at = s;
    if (a.ld_index != a.top_k) {
        const uint32_t k = (uint32_t)a.top_k, t = s / k;
        at = (int64_t)t * a.ld_index + (s - t * k);
    }
    const I v = ((const I *)a.index)[at];
    return v >= 0 && v < a.groups ? (int32_t)v : a.groups;
}

constexpr int SORT_T = 1024, SORT_W = SORT_T / 64;

// Any number of slots in one launch without scratch memory.  Workgroup c
// places the slots of chunk c.  It counts all slots by group itself, those
// before its chunk apart from the rest, which gives every group's first free
// place; then its wavefronts take their 64 slots in turn, a slot's rank
// inside the wavefront from ballots over the bits of the group.
//
// Up to some 16384 slots that count, out of the L2, costs no more than a
// second launch would (in a graph 4096 slots take 6.6 us, 16384 9.1; an empty
// kernel takes 2.4).  Beyond, slots times workgroups bound it: 32768 slots
// 12.5 us, 65536 19.3, 262144 60, 1048576 356, where a launch that counts every
// chunk once and one that places would read the indexes twice; not built.
//
// The counters: `copies` of each, lane l counting in copy l mod copies, so
// that the lanes of a wavefront rarely add to one address.
template <typename I>
__global__ __launch_bounds__(SORT_T) void sort_kernel(DispatchArgs a, int32_t chunk, int32_t copies)
{
    extern __shared__ int32_t counters[];
    const int32_t G = a.groups;
    const uint32_t S = (uint32_t)a.slots;
    int32_t *before = counters, *rest = before + G * copies, *base = rest + G * copies;
    int32_t *sums = base + G;                       // one per wavefront
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t first = blockIdx.x * (uint32_t)chunk;
    const uint32_t last = S - first < (uint32_t)chunk ? S : first + (uint32_t)chunk;
    for (int i = tid; i < 2 * G * copies; i += SORT_T)
        counters[i] = 0;
    __syncthreads();

    constexpr int U = 8;                            // loads in flight per lane
    const int copy = lane & (copies - 1);
    for (uint32_t s0 = 0; s0 < S; s0 += U * SORT_T) {
        int32_t e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t s = s0 + u * SORT_T + tid;     // S < 2^31: no wrap
            e[u] = s < S ? slot_group<I>(a, s) : G;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t s = s0 + u * SORT_T + tid;
            if (e[u] < G)
                atomicAdd((s < first ? before : rest) + e[u] * copies + copy, 1);
        }
    }
    __syncthreads();

    int32_t carry = 0;
    for (int g0 = 0; g0 < G; g0 += SORT_T) {
        const int g = g0 + tid;
        int32_t b = 0, n = 0;
        if (g < G) {
            for (int r = 0; r < copies; ++r) {
                const int at = g * copies + ((r + g) & (copies - 1));   // other banks per lane
                b += before[at];
                n += rest[at];
            }
            n += b;
        }
        const int32_t upto = wave_scan_add(n);
        if (lane == 63)
            sums[wave] = upto;
        __syncthreads();
        int32_t below = carry;
        for (int w = 0; w < SORT_W; ++w) {
            below += w < wave ? sums[w] : 0;
            carry += sums[w];
        }
        if (g < G) {
            base[g] = below + upto - n + b;
            if (blockIdx.x == 0)
                a.offsets[g] = below + upto - n;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        a.offsets[G] = carry;
    // rows of no slot
    for (uint32_t i = ((uint32_t)carry > first ? (uint32_t)carry : first) + tid; i < last; i += SORT_T)
        a.order[i] = -1;

    const int bits = 32 - __builtin_clz((uint32_t)G | 1);       // of 0 .. G
    for (uint32_t s0 = first; s0 < last; s0 += SORT_T) {
        const uint32_t s = s0 + tid;
        const int32_t e = s < last ? slot_group<I>(a, s) : G;
        uint64_t same = ~0ull;
        for (int i = 0; i < bits; ++i) {
            const uint64_t set = __ballot((e >> i) & 1);
            same &= (e >> i) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
        int32_t p = -1;
        for (int w = 0; w < SORT_W; ++w) {
            if (w == wave && e < G) {
                p = base[e] + rank;
                if (rank == n - 1)
                    base[e] = p + 1;
            }
            __syncthreads();
        }
        if (s < last) {
            a.place[s] = p;
            if (p >= 0)
                a.order[p] = (int32_t)s;
        }
    }
}

// 16 bytes of a row, or its last `n` < 16 bytes by elements.
__device__ __forceinline__ void copy_tail(char *dst, const char *src, int n, int elem)
{
    for (int i = 0; i < n; i += elem) {
        if (elem == 4)
            *(uint32_t *)(dst + i) = *(const uint32_t *)(src + i);
        else
            *(uint16_t *)(dst + i) = *(const uint16_t *)(src + i);
    }
}

constexpr int FEW_T = 256;

// Few slots: maps and rows in one launch.  A workgroup has up to KB slots of
// one token.  It counts the slots before each in the sorted order (all S of
// them pass through it once), writes their places and copies the row there,
// whose first pieces are loaded before the count.  The last workgroup writes
// the offsets and the end of order.
template <typename I, int KB>
__global__ __launch_bounds__(FEW_T) void dispatch_few_kernel(DispatchArgs a)
{
    extern __shared__ int32_t count[];              // of the groups; last workgroup
    __shared__ int32_t sums[FEW_T / 64], parts[KB][FEW_T / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t S = a.slots, G = a.groups;
    if (blockIdx.x + 1 < gridDim.x) {
        const uint32_t per = ((uint32_t)a.top_k + KB - 1) / KB;       // workgroups of a token
        const int32_t t = (int32_t)(blockIdx.x / per), j0 = (int32_t)(blockIdx.x - t * per) * KB;
        const char *src = a.x + (int64_t)t * a.ldx;
        constexpr int HELD = 2;
        Raw16 held[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int64_t at = (int64_t)(u * FEW_T + tid) * 16;
            if (at + 16 <= a.width)
                held[u] = load_raw16(src + at);
        }
        const int32_t b = t * a.top_k + j0;     // its first slot
        int32_t e[KB], n[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            e[j] = j0 + j < a.top_k ? slot_group<I>(a, (uint32_t)(b + j)) : G;
            n[j] = 0;
        }
        constexpr int U = 4;                    // loads in flight
        for (int32_t s0 = 0; s0 < S; s0 += U * FEW_T) {
            int32_t v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t s = s0 + u * FEW_T + tid;
                v[u] = s < S ? slot_group<I>(a, (uint32_t)s) : G;      // before no slot of a group
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t s = s0 + u * FEW_T + tid;
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    n[j] += v[u] < e[j] || (v[u] == e[j] && s < b + j);
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int32_t sum = wave_scan_add(n[j]);
            if (lane == 63)
                parts[j][wave] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (j0 + j >= a.top_k)
                continue;
            if (e[j] >= G) {
                if (tid == 0)
                    a.place[b + j] = -1;
                continue;
            }
            int32_t p = 0;
#pragma unroll
            for (int w = 0; w < FEW_T / 64; ++w)
                p += parts[j][w];
            if (tid == 0) {
                a.place[b + j] = p;
                a.order[p] = b + j;
            }
            char *dst = a.rows + (int64_t)p * a.ldr;
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                const int64_t at = (int64_t)(u * FEW_T + tid) * 16;
                if (at + 16 <= a.width)
                    store_raw16(dst + at, held[u]);
            }
            for (int64_t at = (int64_t)(HELD * FEW_T + tid) * 16; at + 16 <= a.width; at += FEW_T * 16)
                store_raw16(dst + at, load_raw16(src + at));
            const int64_t whole = a.width & ~(int64_t)15;
            if (tid == 0)
                copy_tail(dst + whole, src + whole, (int)(a.width - whole), a.elem);
        }
        return;
    }
    for (int i = tid; i < G; i += FEW_T)
        count[i] = 0;
    __syncthreads();
    for (int32_t s = tid; s < S; s += FEW_T) {
        const int32_t e = slot_group<I>(a, (uint32_t)s);
        if (e < G)
            atomicAdd(count + e, 1);
    }
    __syncthreads();
    int32_t carry = 0;
    for (int g0 = 0; g0 < G; g0 += FEW_T) {
        const int g = g0 + tid;
        const int32_t n = g < G ? count[g] : 0;
        const int32_t upto = wave_scan_add(n);
        if (lane == 63)
            sums[wave] = upto;
        __syncthreads();
        int32_t below = carry;
#pragma unroll
        for (int w = 0; w < FEW_T / 64; ++w) {
            below += w < wave ? sums[w] : 0;
            carry += sums[w];
        }
        if (g < G)
            a.offsets[g] = below + upto - n;
        __syncthreads();
    }
    if (tid == 0)
        a.offsets[G] = carry;
    for (int32_t i = carry + tid; i < S; i += FEW_T)
        a.order[i] = -1;
}

// A wavefront takes 64 x U pieces of 16 bytes of one token's row and writes
// them to each of its places: x is read once, whatever top_k is.
constexpr int SPREAD_U = 2, SPREAD_T = 256;

__global__ __launch_bounds__(SPREAD_T) void spread_kernel(SpreadArgs a)
{
    constexpr int64_t SEG = 64 * SPREAD_U * 16;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t segs = (uint32_t)((a.width + SEG - 1) / SEG);
    const int64_t units = a.tokens * segs, step = (int64_t)gridDim.x * (SPREAD_T / 64);
    for (int64_t unit = (int64_t)blockIdx.x * (SPREAD_T / 64) + wave; unit < units; unit += step) {
        const int64_t t = unit / segs, first = (unit - t * segs) * SEG;
        const char *src = a.x + t * a.ldx;
        Raw16 v[SPREAD_U];
#pragma unroll
        for (int u = 0; u < SPREAD_U; ++u) {
            const int64_t at = first + (u * 64 + lane) * 16;
            if (at + 16 <= a.width)
                v[u] = load_raw16(src + at);
        }
        for (int32_t j = 0; j < a.top_k; ++j) {
            const int32_t p = a.place[t * a.top_k + j];
            if (p < 0 || p >= a.limit)
                continue;
            char *dst = a.rows + (int64_t)p * a.ldr;
#pragma unroll
            for (int u = 0; u < SPREAD_U; ++u) {
                const int64_t at = first + (u * 64 + lane) * 16;
                if (at + 16 <= a.width)
                    store_raw16(dst + at, v[u]);
                else if (at < a.width)
                    copy_tail(dst + at, src + at, (int)(a.width - at), a.elem);
            }
        }
    }
}

template <int KB>
void launch_few(const DispatchArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)(a.slots / a.top_k * ((a.top_k + KB - 1) / KB)) + 1);
    const size_t lds = (size_t)a.groups * 4;
    if (a.index_bits == 64)
        hipLaunchKernelGGL((dispatch_few_kernel<int64_t, KB>), grid, dim3(FEW_T), lds, s, a);
    else
        hipLaunchKernelGGL((dispatch_few_kernel<int32_t, KB>), grid, dim3(FEW_T), lds, s, a);
}

} // namespace

hipError_t launch_dispatch_sort(const DispatchArgs &a, hipStream_t s)
{
    // chunks of whole rounds of the workgroup, at most 256 of them
    const int64_t rounds = ((int64_t)a.slots + 256 * SORT_T - 1) / (256 * SORT_T);
    const int64_t chunk = SORT_T * (rounds < 1 ? 1 : rounds);
    int32_t copies = 32;
    while (copies > 1 && (int64_t)a.groups * copies > kMaxDispatchGroups)
        copies /= 2;
    const size_t lds = ((size_t)2 * a.groups * copies + a.groups + SORT_W) * 4;
    const dim3 grid((unsigned)(a.slots > 0 ? (a.slots + chunk - 1) / chunk : 1));
    if (a.index_bits == 64)
        hipLaunchKernelGGL(sort_kernel<int64_t>, grid, dim3(SORT_T), lds, s, a, (int32_t)chunk, copies);
    else
        hipLaunchKernelGGL(sort_kernel<int32_t>, grid, dim3(SORT_T), lds, s, a, (int32_t)chunk, copies);
    return hipGetLastError();
}

hipError_t launch_dispatch_few(const DispatchArgs &a, hipStream_t s)
{
    // two slots a workgroup from 1024 on, where the counting bounds it (1024
    // slots, 2 a token, 2048 bf16: 4.4 us with one, 4.6 with two; 2048 slots
    // 7.4 and 6.5)
    if (a.top_k == 1 || a.slots <= 1024)
        launch_few<1>(a, s);
    else
        launch_few<2>(a, s);
    return hipGetLastError();
}

hipError_t launch_spread(const SpreadArgs &a, hipStream_t s)
{
    constexpr int64_t SEG = 64 * SPREAD_U * 16;
    const int64_t groups = (a.tokens * ((a.width + SEG - 1) / SEG) + SPREAD_T / 64 - 1) / (SPREAD_T / 64);
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : 1 << 20));
    hipLaunchKernelGGL(spread_kernel, grid, dim3(SPREAD_T), 0, s, a);
    return hipGetLastError();
}

} // namespace dg
