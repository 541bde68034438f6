// norm.hip -- root-mean-square norm with the residual's addition, and its
// gradient:
//
//   h = x + residual, rounded to their type (what the gradient reads again)
//   r = 1 / sqrt(sum h^2 / k + eps)
//   y = h r w                 rounded once, and / or as E4M3 codes with a
//                             float32 scale for each 128 columns (quant.hip's)
//   g = dy w
//   dx = r (g - h r^2 sum(g h) / k) + dh        (dh: the gradient of h itself)
//   dw = sum over rows of dy h r
//
// Rows are read once: a workgroup (or a wave) holds a row in registers
// between its sum and its output.  Everything is computed in float32.
#include "device.hpp"
#include "layers.hpp"
#include "rows.hpp"

namespace agg {

namespace {

template <int kType>
constexpr int elt_bytes() { return kType == kTypeF32 ? 4 : 2; }

// The sum over a workgroup's threads, in all of them: lanes, then waves in
// order.  `slot`: float[kWaves], not in use by a sum that some wave may still
// be reading (callers alternate between two).
template <int kWaves>
__device__ __forceinline__ float group_sum(float v, float* slot)
{
    v = wave_sum(v);
    if constexpr (kWaves == 1) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += slot[w];
    return v;
}

// x + res in float32, rounded to kType's values.
template <int kType>
__device__ __forceinline__ void add_rounded(float (&v)[8], const float (&r)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen<kType>(narrow_bits<kType>(v[e] + r[e]));
}

__device__ __forceinline__ float rstd_of(float sum, const NormArgs& a)
{
    return 1.f / sqrtf(sum / (float)a.k + a.eps);
}

// A lane's eight columns as E4M3 codes, and by the first of 16 lanes their block's
// scale.  y / amax(y) = u / amax(u) with u = h w, which is exact for 16-bit
// types: the code does not need r and its roundings.  448 u / amax(u) is then
// corrected by what the division and the product rounded off, so that a code is
// another than the exact value's only within 2^-24 of a tie.  Blocks at the ends
// of the range (zeros, the floor, infinities, NaN) go by y itself.
template <bool kWide>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t row, int64_t col, const float (&h)[8],
                                            const float (&w)[8], float rstd)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = h[e] * w[e];
    uint32_t m = max16(max_bits(v));
    float amax = __builtin_bit_cast(float, m);
    const uint32_t top = __builtin_bit_cast(uint32_t, amax * rstd);
    if (m > kAmaxFloor && m < 0x7f800000u && top > kAmaxFloor && top < 0x7f800000u) {
        const float inverse = kE4M3Max / amax;
        const float rest = fmaf(-inverse, amax, kE4M3Max) / kE4M3Max;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float r = v[e] * inverse;
            v[e] = r + fmaf(r, rest, fmaf(v[e], inverse, -r));
        }
        store8<kWide>(a.q + row * a.ldq, col, a.k, v, 1.f);
        amax = __builtin_bit_cast(float, top);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = h[e] * rstd * w[e];
        m = max16(max_bits(v));
        amax = __builtin_bit_cast(float, m > kAmaxFloor ? m : kAmaxFloor);
        store8<kWide>(a.q + row * a.ldq, col, a.k, v, kE4M3Max / amax);
    }
    if (threadIdx.x % 16 == 0 && col < a.k) a.scale[row * a.lds + col / kScaleBlock] = amax / kE4M3Max;
}

// kPer pieces of eight columns a thread, the row's pieces dealt to the
// threads in turn.  The weight is loaded with the row: behind the sum it would
// be another memory latency.
template <int kType, int kThreads, int kPer>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a)
{
    constexpr int kWaves = kThreads / 64, kElt = elt_bytes<kType>();
    __shared__ float slot[2][kWaves];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        Raw8<kType> x[kPer], r[kPer], w[kPer];
        float v[kPer][8];
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = (u * kThreads + (int)threadIdx.x) * 8;
            x[u].load(a.x + row * a.ldx * kElt, col, a.k);
            if (a.res) r[u].load(a.res + row * a.ldr * kElt, col, a.k);
        }
        if (a.weight)
#pragma unroll
            for (int u = 0; u < kPer; ++u) w[u].load(a.weight, (u * kThreads + (int)threadIdx.x) * 8, a.k);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = x[u][e];
            if (a.res)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[u][e] = widen<kType>(narrow_bits<kType>(v[u][e] + r[u][e]));
        }
        if (a.h)
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                store_row8<kType, true>(a.h + row * a.ldh * kElt, (u * kThreads + (int)threadIdx.x) * 8, a.k, v[u]);
#pragma unroll
        for (int u = 0; u < kPer; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[u][e] * v[u][e];
        const float rstd = rstd_of(group_sum<kWaves>(sum, slot[turn]), a);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = (u * kThreads + (int)threadIdx.x) * 8;
            float f[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = a.weight ? w[u][e] : 1.f;
                y[e] = v[u][e] * rstd * f[e];
            }
            if (a.y) store_row8<kType, true>(a.y + row * a.ldy * kElt, col, a.k, y);
            // 16 lanes a block of 128; all lanes of a wave are here
            if (a.q) store_codes<true>(a, row, col, v[u], f, rstd);
        }
    }
}

// Any length and alignment: the row is walked twice, h or what it is made of
// being read again by the thread that read (and wrote) it before.
template <int kType>
__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs a)
{
    constexpr int kElt = elt_bytes<kType>();
    __shared__ float slot[2][4];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const char* x = a.x + row * a.ldx * kElt;
        const char* res = a.res ? a.res + row * a.ldr * kElt : nullptr;
        char* h = a.h ? a.h + row * a.ldh * kElt : nullptr;
        float sum = 0.f;
        for (int64_t c0 = 0; c0 < a.k; c0 += 2048) {
            const int64_t col = c0 + threadIdx.x * 8;
            float v[8];
            load8<kType, false>(x, col, a.k, v);
            if (res) {
                float r[8];
                load8<kType, false>(res, col, a.k, r);
                add_rounded<kType>(v, r);
            }
            if (h) store_row8<kType, false>(h, col, a.k, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[e] * v[e];
        }
        const float rstd = rstd_of(group_sum<4>(sum, slot[turn]), a);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        for (int64_t c0 = 0; c0 < a.k; c0 += 2048) {
            const int64_t col = c0 + threadIdx.x * 8;
            float v[8], w[8];
            if (h) {
                load8<kType, false>(h, col, a.k, v);     // h may be x or res, which it has replaced
            } else {
                load8<kType, false>(x, col, a.k, v);
                if (res) {
                    float r[8];
                    load8<kType, false>(res, col, a.k, r);
                    add_rounded<kType>(v, r);
                }
            }
            if (a.weight) load8<kType, false>(a.weight, col, a.k, w);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!a.weight) w[e] = 1.f;
                y[e] = v[e] * rstd * w[e];
            }
            if (a.y) store_row8<kType, false>(a.y + row * a.ldy * kElt, col, a.k, y);
            if (a.q) store_codes<false>(a, row, col, v, w, rstd);
        }
    }
}

// ---- gradient -----------------------------------------------------------------
//
// A workgroup walks every gridDim.x-th row, the next one's loads under way while
// this one is summed, and keeps its part of the weight's gradient, which
// norm_join_kernel adds over the workgroups in order.

template <int kType, int kThreads, int kPer>
__global__ __launch_bounds__(kThreads) void norm_grad_kernel(NormGradArgs a)
{
    constexpr int kWaves = kThreads / 64, kElt = elt_bytes<kType>();
    __shared__ float slot[2][kWaves];
    struct Row {
        Raw8<kType> dy[kPer], h[kPer], dh[kPer];
        float rstd;
    };
    const auto load = [&](Row& r, int64_t row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = (u * kThreads + (int)threadIdx.x) * 8;
            r.dy[u].load(a.dy + row * a.lddy * kElt, col, a.k);
            r.h[u].load(a.h + row * a.ldh * kElt, col, a.k);
            if (a.dh) r.dh[u].load(a.dh + row * a.lddh * kElt, col, a.k);
        }
        r.rstd = a.rstd[row];
    };
    Raw8<kType> w[kPer];
    float dw[kPer][8] = {};
    Row now, next;
    load(now, blockIdx.x);
    if (a.weight)
#pragma unroll
        for (int u = 0; u < kPer; ++u) w[u].load(a.weight, (u * kThreads + (int)threadIdx.x) * 8, a.k);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        load(next, row + gridDim.x);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < kPer; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dy = now.dy[u][e], h = now.h[u][e];
                dw[u][e] += dy * (h * now.rstd);
                sum += (a.weight ? dy * w[u][e] : dy) * h;
            }
        const float c = group_sum<kWaves>(sum, slot[turn]) / (float)a.k * now.rstd * now.rstd;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = (u * kThreads + (int)threadIdx.x) * 8;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dy = now.dy[u][e], h = now.h[u][e];
                const float dx = now.rstd * ((a.weight ? dy * w[u][e] : dy) - h * c);
                d[e] = a.dh ? dx + now.dh[u][e] : dx;
            }
            store_row8<kType, true>(a.dx + row * a.lddx * kElt, col, a.k, d);
        }
        now = next;
    }
    if (!a.dw) return;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int col = (u * kThreads + (int)threadIdx.x) * 8;
        if (col < a.k) store_row8<kTypeF32, true>(reinterpret_cast<char*>(a.partial + blockIdx.x * a.k), col, a.k, dw[u]);
    }
}

// Any length and alignment; the workgroup's part of the weight's gradient
// lives in memory, each thread adding to the columns that are its own.
template <int kType>
__global__ __launch_bounds__(256) void norm_grad_any_kernel(NormGradArgs a)
{
    constexpr int kElt = elt_bytes<kType>();
    __shared__ float slot[2][4];
    float* part = a.dw ? a.partial + blockIdx.x * a.k : nullptr;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const char* dy = a.dy + row * a.lddy * kElt;
        const char* h = a.h + row * a.ldh * kElt;
        const float rstd = a.rstd[row];
        const bool first = row == blockIdx.x;
        float sum = 0.f;
        for (int64_t c0 = 0; c0 < a.k; c0 += 2048) {
            const int64_t col = c0 + threadIdx.x * 8;
            float g[8], v[8], w[8];
            load8<kType, false>(dy, col, a.k, g);
            load8<kType, false>(h, col, a.k, v);
            if (a.weight) load8<kType, false>(a.weight, col, a.k, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (part && col + e < a.k) {
                    const float p = g[e] * (v[e] * rstd);
                    part[col + e] = first ? p : part[col + e] + p;
                }
                sum += (a.weight ? g[e] * w[e] : g[e]) * v[e];
            }
        }
        const float c = group_sum<4>(sum, slot[turn]) / (float)a.k * rstd * rstd;
        for (int64_t c0 = 0; c0 < a.k; c0 += 2048) {
            const int64_t col = c0 + threadIdx.x * 8;
            float g[8], v[8], w[8], d[8];
            load8<kType, false>(dy, col, a.k, g);
            load8<kType, false>(h, col, a.k, v);
            if (a.weight) load8<kType, false>(a.weight, col, a.k, w);
            if (a.dh) load8<kType, false>(a.dh + row * a.lddh * kElt, col, a.k, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dx = rstd * ((a.weight ? g[e] * w[e] : g[e]) - v[e] * c);
                d[e] = a.dh ? dx + d[e] : dx;
            }
            store_row8<kType, false>(a.dx + row * a.lddx * kElt, col, a.k, d);
        }
    }
}

// dw[c] = the sum of partial[p][c] over p: 32 columns and 32 shares of the
// parts a workgroup, the shares then in order.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormGradArgs a)
{
    __shared__ float lds[32][33];
    const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + c;
    float sum = 0.f;
    if (col < a.k)
#pragma unroll 8
        for (int p = s; p < a.parts; p += 32) sum += a.partial[p * a.k + col];
    lds[s][c] = sum;
    __syncthreads();
    if (s || col >= a.k) return;
#pragma unroll
    for (int u = 1; u < 32; ++u) sum += lds[u][c];
    if (a.dw_type == kTypeF32) reinterpret_cast<float*>(a.dw)[col] = sum;
    else reinterpret_cast<uint16_t*>(a.dw)[col] = to_bits16(sum, a.dw_type);
}

constexpr int64_t kMaxRowsAtOnce = 1 << 21;     // workgroups of at most 1024 threads

template <int kType>
hipError_t launch_norm_of(const NormArgs& a, bool wide, hipStream_t st)
{
    const dim3 grid((uint32_t)(a.rows < kMaxRowsAtOnce ? a.rows : kMaxRowsAtOnce));
    if (!wide || a.k > 16384) hipLaunchKernelGGL((norm_any_kernel<kType>), grid, dim3(256), 0, st, a);
    else if (a.k <= 512) hipLaunchKernelGGL((norm_kernel<kType, 64, 1>), grid, dim3(64), 0, st, a);
    else if (a.k <= 2048) hipLaunchKernelGGL((norm_kernel<kType, 256, 1>), grid, dim3(256), 0, st, a);
    else if (a.k <= 4096) hipLaunchKernelGGL((norm_kernel<kType, 256, 2>), grid, dim3(256), 0, st, a);
    else if (a.k <= 8192) hipLaunchKernelGGL((norm_kernel<kType, 1024, 1>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((norm_kernel<kType, 1024, 2>), grid, dim3(1024), 0, st, a);
    return hipGetLastError();
}

// Past 8192 columns a row and the next no longer fit the registers of one
// workgroup's 512 threads, and rows are read element by element: 4096 rows of 8192
// bf16 take 61 us (4.4 TB/s), of 12288 617, of 16384 802 (the forward kernels 51,
// 84 and 109).
template <int kType>
hipError_t launch_norm_grad_of(const NormGradArgs& a, bool wide, hipStream_t st)
{
    const dim3 grid((uint32_t)a.parts);
    if (a.rows > 0) {
        if (!wide || a.k > 8192) hipLaunchKernelGGL((norm_grad_any_kernel<kType>), grid, dim3(256), 0, st, a);
        else if (a.k <= 2048) hipLaunchKernelGGL((norm_grad_kernel<kType, 256, 1>), grid, dim3(256), 0, st, a);
        else if (a.k <= 4096) hipLaunchKernelGGL((norm_grad_kernel<kType, 256, 2>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((norm_grad_kernel<kType, 512, 2>), grid, dim3(512), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.dw) return e;
    }
    if (!a.dw) return hipSuccess;
    hipLaunchKernelGGL(norm_join_kernel, dim3((uint32_t)((a.k + 31) / 32)), dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int type, bool wide, hipStream_t st)
{
    if (type == kTypeF32) return launch_norm_of<kTypeF32>(a, wide, st);
    return type == kTypeF16 ? launch_norm_of<kTypeF16>(a, wide, st) : launch_norm_of<kTypeBF16>(a, wide, st);
}

hipError_t launch_norm_grad(const NormGradArgs& a, int type, bool wide, hipStream_t st)
{
    if (type == kTypeF32) return launch_norm_grad_of<kTypeF32>(a, wide, st);
    return type == kTypeF16 ? launch_norm_grad_of<kTypeF16>(a, wide, st)
                            : launch_norm_grad_of<kTypeBF16>(a, wide, st);
}

}  // namespace agg
