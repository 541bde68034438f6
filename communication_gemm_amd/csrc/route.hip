// route.hip -- tokens sorted by the experts they go to, and back.
//
//   sort      offsets[e] = number of assignments with an expert below e
//             place[f] = offsets[e] + number of earlier assignments of e
//   dispatch  xs[place[t, j]] = x[t]
//   combine   y[t] = sum_j w[t, j] h[place[t, j]]
//   gradient  dh[place[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], h[place[t, j]]>
//
// All but the sort go by tokens: a token's row is read (or written) once
// whatever `top` is, and its places come through scalar loads.
#include <atomic>

#include "device.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "layers.hpp"
#include "rows.hpp"

namespace agg {

namespace {

// ---- sort -----------------------------------------------------------------
//
// A counting sort whose order depends only on the input.  Workgroup b places
// the b-th chunk of assignments; its waves take a stretch each.  Where an
// expert's assignments of a stretch begin follows from the counts of all
// chunks before it and of the stretches before it in its own chunk; within
// 64 assignments the rank is a count of equal lanes below, from one ballot
// for each bit of the expert's number.

template <class Id>
__device__ __forceinline__ int expert_of(const SortArgs& a, uint32_t f)
{
    int64_t at = f;
    if (a.ld != a.top) {
        const uint32_t t = f / (uint32_t)a.top;
        at = (int64_t)t * a.ld + (f - t * (uint32_t)a.top);
    }
    const Id v = static_cast<const Id*>(a.ids)[at];
    return v >= 0 && v < (Id)a.experts ? (int)v : -1;
}

// f(assignment, expert) for the assignments lo .. hi that have one, a stride of
// kThreads apart, kAhead loads at a time (16384 assignments: the sort takes 7.85
// us, 7.90 one load after the other).
constexpr int kAhead = 8;

template <class Id, int kThreads, class F>
__device__ __forceinline__ void for_experts(const SortArgs& a, uint32_t lo, uint32_t hi, F f)
{
    for (uint32_t f0 = lo + threadIdx.x; f0 < hi; f0 += kThreads * kAhead) {
        int e[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t at = f0 + u * kThreads;
            e[u] = at < hi ? expert_of<Id>(a, at) : -1;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (e[u] >= 0) f(f0 + u * kThreads, e[u]);
    }
}

template <class Id>
__global__ __launch_bounds__(1024) void sort_count_kernel(SortArgs a)
{
    extern __shared__ int count[];
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) count[e] = 0;
    __syncthreads();
    const uint32_t c0 = blockIdx.x * (uint32_t)a.chunk;
    const uint32_t c1 = min((uint32_t)a.n, c0 + (uint32_t)a.chunk);
    for_experts<Id, 1024>(a, c0, c1, [&](uint32_t, int e) { atomicAdd(count + e, 1); });
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// kCounted: the chunks' counts are in a.counts; otherwise every workgroup
// counts all assignments itself.
template <class Id, int kThreads, bool kCounted>
__global__ __launch_bounds__(kThreads) void sort_place_kernel(SortArgs a)
{
    constexpr int kWaves = kThreads / 64;
    extern __shared__ int lds[];
    __shared__ uint32_t sums[kWaves];
    const int E = a.experts;
    int* before = lds;               // of the chunks before this one
    int* after = before + E;
    int* own = after + E;            // [kWaves][E] of this chunk's stretches, then their next places
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    for (int u = threadIdx.x; u < (kWaves + 2) * E; u += kThreads) lds[u] = 0;
    __syncthreads();
    const uint32_t n = (uint32_t)a.n, chunk = (uint32_t)a.chunk, stretch = chunk / kWaves;
    const uint32_t c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
    if constexpr (kCounted)
        // a thread adds one expert's counts of every rows-th chunk
        for (int e0 = 0; e0 < E; e0 += kThreads) {
            const int width = min(E - e0, kThreads), rows = kThreads / width;
            const int e = e0 + (int)threadIdx.x % width, b0 = (int)threadIdx.x / width;
            int lower = 0, upper = 0;
            if (b0 < rows)
#pragma unroll 8
                for (int b = b0; b < (int)gridDim.x; b += rows) {
                    const int v = a.counts[(int64_t)b * E + e];
                    lower += b < (int)blockIdx.x ? v : 0;
                    upper += b > (int)blockIdx.x ? v : 0;
                }
            if (lower) atomicAdd(before + e, lower);
            if (upper) atomicAdd(after + e, upper);
        }
    for_experts<Id, kThreads>(a, kCounted ? c0 : 0, kCounted ? c1 : n, [&](uint32_t f, int e) {
        atomicAdd((f < c0 ? before : f >= c1 ? after : own + (f - c0) / stretch * E) + e, 1);
    });
    __syncthreads();
    uint32_t carry = 0;
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + (int)threadIdx.x;
        uint32_t total = 0;
        if (e < E) {
            total = (uint32_t)(before[e] + after[e]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) total += (uint32_t)own[w * E + e];
        }
        uint32_t sum = wave_inclusive_sum(total);
        if (e0) __syncthreads();     // everyone has read the last part's sums
        if (lane == 63) sums[wave] = sum;
        __syncthreads();
        uint32_t part = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) sum += sums[w];
            part += sums[w];
        }
        if (e < E) {
            const uint32_t start = carry + sum - total;
            if (blockIdx.x == 0) a.offsets[e] = (int)start;
            int next = (int)start + before[e];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int c = own[w * E + e];
                own[w * E + e] = next;
                next += c;
            }
        }
        carry += part;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = (int)carry;
    __syncthreads();
    volatile int* mine = own + wave * E;
    const int bits = 32 - __builtin_clz((unsigned)E);     // also of E itself, the number of no expert
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (uint32_t s = 0; s < stretch; s += 64) {
        const uint32_t f0 = c0 + (uint32_t)wave * stretch + s, f = f0 + (uint32_t)lane;
        if (f0 >= c1) break;
        int e = f < c1 ? expert_of<Id>(a, f) : -1;
        const bool has = e >= 0;
        e = has ? e : E;
        uint64_t same = ~(uint64_t)0;
        for (int b = 0; b < bits; ++b) {
            const bool set = (e >> b) & 1;
            const uint64_t vote = __builtin_amdgcn_ballot_w64(set);
            same &= set ? vote : ~vote;
        }
        const int rank = __builtin_popcountll(same & below);
        const int at = has ? mine[e] : 0;
        if (f < c1) a.place[f] = has ? at + rank : -1;
        // a wave's LDS accesses stay in order: every lane has read by now
        if (has && rank == 0) mine[e] = at + __builtin_popcountll(same);
    }
}

template <class Id, int kThreads>
hipError_t launch_place(const SortArgs& a, hipStream_t st)
{
    const int lds = (kThreads / 64 + 2) * a.experts * 4;
    const uint32_t blocks = (uint32_t)sort_blocks(a.n);
    const bool counted = a.n > kSortRecount;
    static std::atomic<uint64_t> done[2];
    const auto kernel = counted ? sort_place_kernel<Id, kThreads, true> : sort_place_kernel<Id, kThreads, false>;
    if (lds > 60 * 1024) {
        const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), 160 * 1024 - 256, done[counted]);
        if (e != hipSuccess) return e;
    }
    if (counted) {
        hipLaunchKernelGGL((sort_count_kernel<Id>), dim3(blocks), dim3(1024), a.experts * 4, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), lds, st, a);
    return hipGetLastError();
}

template <class Id>
hipError_t launch_sort_of(const SortArgs& a, hipStream_t st)
{
    // four waves where a chunk has no work for more, or sixteen waves' counts
    // would not fit
    return a.n <= 256 || a.experts > 2048 ? launch_place<Id, 256>(a, st) : launch_place<Id, 1024>(a, st);
}

// ---- dispatch ---------------------------------------------------------------

// Whether a place names a row.
__device__ __forceinline__ bool is_row(int p, int rows) { return p >= 0 && p < rows; }

template <class U>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs a)
{
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * sizeof(U);
    if (col >= a.row_bytes) return;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const U v = *reinterpret_cast<const U*>(a.x + t * a.ldx + col);
        const int32_t* place = a.place + t * a.top;
        for (int j = 0; j < a.top; ++j) {
            const int p = place[j];
            if (is_row(p, a.rows)) *reinterpret_cast<U*>(a.xs + p * a.ldxs + col) = v;
        }
    }
}

// Threads of a workgroup (whole waves, at most 256) that share a row of
// `units`, and the grid: tokens (a stride apart where they are too many) and
// parts of a row.
struct RowGrid {
    dim3 grid, threads;
};

inline RowGrid row_grid(int64_t tokens, int64_t units)
{
    const int64_t threads = units >= 256 ? 256 : (units + 63) / 64 * 64;
    const int64_t x = tokens < (1 << 23) ? tokens : (1 << 23);
    return {dim3((uint32_t)x, (uint32_t)((units + threads - 1) / threads)), dim3((uint32_t)threads)};
}

template <class U>
hipError_t launch_dispatch_of(const DispatchArgs& a, hipStream_t st)
{
    const RowGrid g = row_grid(a.tokens, (a.row_bytes + sizeof(U) - 1) / sizeof(U));
    hipLaunchKernelGGL((dispatch_kernel<U>), g.grid, g.threads, 0, st, a);
    return hipGetLastError();
}

// ---- combine ----------------------------------------------------------------

constexpr int kAtOnce = 4;     // rows of h under way a lane

template <int kType, int kOut, bool kWide>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2, kOutElt = kOut == kTypeF32 ? 4 : 2;
    const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 8;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float acc[8] = {};
        for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
            float v[kAtOnce][8], w[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int j = j0 + u;
                const int p = j < a.top ? a.place[t * a.top + j] : -1;
                const bool in = is_row(p, a.rows);      // rows of no place add nothing, whatever their weight
                w[u] = in ? a.w ? a.w[t * a.ldw + j] : 1.f : 0.f;
                load8<kType, kWide>(a.h + (in ? p : 0) * a.ldh * kElt, col, in ? a.k : 0, v[u]);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += w[u] * v[u][e];
        }
        store_row8<kOut, kWide>(a.y + t * a.ldy * kOutElt, col, a.k, acc);
    }
}

// A workgroup a token.  The weights' gradients are sums over the row: each
// lane's columns, then the lanes, then the waves in their order.
template <int kType, bool kWide>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    __shared__ float part[4][kAtOnce];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
        for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
            int p[kAtOnce];
            float w[kAtOnce], sum[kAtOnce] = {};
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                p[u] = j0 + u < a.top ? a.place[t * a.top + j0 + u] : -1;
                if (!is_row(p[u], a.rows)) p[u] = -1;
                w[u] = p[u] >= 0 ? a.w[t * a.ldw + j0 + u] : 0.f;
            }
            for (int64_t c0 = 0; c0 < a.k; c0 += blockDim.x * 8) {
                const int64_t col = c0 + threadIdx.x * 8;
                float dy[8], h[kAtOnce][8];
                load8<kType, kWide>(a.y + t * a.ldy * kElt, col, a.k, dy);
                if (a.dw)
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        load8<kType, kWide>(a.h + (p[u] < 0 ? 0 : p[u]) * a.ldh * kElt, col,
                                            p[u] < 0 ? 0 : a.k, h[u]);
                if (a.dh)
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        if (p[u] >= 0) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = w[u] * dy[e];
                            store_row8<kType, kWide>(a.dh + p[u] * a.lddh * kElt, col, a.k, v);
                        }
                if (a.dw)
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[u] += dy[e] * h[u][e];
            }
            if (!a.dw) continue;
            __syncthreads();       // the last sums have been read
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const float s = wave_sum(sum[u]);
                if (lane == 0) part[wave][u] = s;
            }
            __syncthreads();
            const int j = j0 + (int)threadIdx.x;
            if (threadIdx.x < kAtOnce && j < a.top) {
                float s = part[0][threadIdx.x];
                for (int v = 1; v < waves; ++v) s += part[v][threadIdx.x];
                // no place: no product, whatever dy and h hold
                a.dw[t * a.lddw + j] = is_row(a.place[t * a.top + j], a.rows) ? s : 0.f;
            }
        }
}

template <int kType, int kOut>
hipError_t launch_combine_of(const CombineArgs& a, bool wide, hipStream_t st)
{
    const RowGrid g = row_grid(a.tokens, (a.k + 7) / 8);
    const auto kernel = wide ? combine_kernel<kType, kOut, true> : combine_kernel<kType, kOut, false>;
    hipLaunchKernelGGL(kernel, g.grid, g.threads, 0, st, a);
    return hipGetLastError();
}

template <int kType>
hipError_t launch_combine_grad_of(const CombineArgs& a, bool wide, hipStream_t st)
{
    const RowGrid g = row_grid(a.tokens, (a.k + 7) / 8);
    const auto kernel = wide ? combine_grad_kernel<kType, true> : combine_grad_kernel<kType, false>;
    hipLaunchKernelGGL(kernel, dim3(g.grid.x), g.threads, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, bool wide_ids, hipStream_t st)
{
    return wide_ids ? launch_sort_of<int64_t>(a, st) : launch_sort_of<int32_t>(a, st);
}

// unit: bytes a lane moves at a time, 16 or an element.
hipError_t launch_dispatch(const DispatchArgs& a, int unit, hipStream_t st)
{
    if (unit == 16) return launch_dispatch_of<uint4>(a, st);
    if (unit == 4) return launch_dispatch_of<uint32_t>(a, st);
    return unit == 2 ? launch_dispatch_of<uint16_t>(a, st) : launch_dispatch_of<uint8_t>(a, st);
}

hipError_t launch_combine(const CombineArgs& a, int type, int out_type, bool wide, hipStream_t st)
{
    if (type == kTypeF32) return launch_combine_of<kTypeF32, kTypeF32>(a, wide, st);
    if (type == kTypeF16)
        return out_type == kTypeF32 ? launch_combine_of<kTypeF16, kTypeF32>(a, wide, st)
                                    : launch_combine_of<kTypeF16, kTypeF16>(a, wide, st);
    return out_type == kTypeF32 ? launch_combine_of<kTypeBF16, kTypeF32>(a, wide, st)
                                : launch_combine_of<kTypeBF16, kTypeBF16>(a, wide, st);
}

hipError_t launch_combine_grad(const CombineArgs& a, int type, bool wide, hipStream_t st)
{
    if (type == kTypeF32) return launch_combine_grad_of<kTypeF32>(a, wide, st);
    return type == kTypeF16 ? launch_combine_grad_of<kTypeF16>(a, wide, st)
                            : launch_combine_grad_of<kTypeBF16>(a, wide, st);
}

}  // namespace agg
