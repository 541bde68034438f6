// mx.hip -- products of microscaled 4-bit codes, dense and by expert:
//
//   c[m, n] = sum over blocks j of 32 k of
//             2^(ea[m, j] + eb[n, j] - 254) * sum over k in j of a[m, k] b[n, k]
#include <atomic>

#include "device.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "layers.hpp"
#include "mx.hpp"

namespace agg {

namespace {

// ---- every layout -------------------------------------------------------
//
// 64 x 64 tiles, four waves of 32 x 32, 256 r (128 bytes) at a time, codes
// loaded byte by byte and scales one by one with all edges checked.

constexpr int kAnyTile = 64;
constexpr int kAnyPitch = 128 + 16;

__device__ __forceinline__ void load_any(char* lds, const char* src, int64_t ld, int rows, int64_t left)
{
#pragma unroll 4
    for (int u = threadIdx.x; u < kAnyTile * 128; u += 256) {
        const int i = u / 128, r = u % 128;
        lds[i * kAnyPitch + r] = i < rows && r < left ? src[i * ld + r] : 0;
    }
}

__global__ __launch_bounds__(256) void mx_any_layout_kernel(MxArgs a)
{
    __shared__ __attribute__((aligned(16))) char lp[kAnyTile * kAnyPitch];
    __shared__ __attribute__((aligned(16))) char lq[kAnyTile * kAnyPitch];
    TileRef t;
    if (!find_tile<kAnyTile, 4>(a, blockIdx.x, (a.J + kAnyTile - 1) / kAnyTile, t)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j0 = t.j * kAnyTile;
    const int cols = a.J - j0 < kAnyTile ? a.J - j0 : kAnyTile;
    const int kb = (a.R + kMxBlock - 1) / kMxBlock;
    const int64_t bytes = a.R / 2;
    const char* p = a.p + t.row0 * a.ldp;
    const char* q = a.q + t.group * a.q_stride + j0 * a.ldq;
    const uint8_t* pe = a.pe + t.row0 * a.ldps;
    const uint8_t* qe = a.qe + t.group * a.qs_stride + j0 * a.ldqs;
    const int wi = (wave & 1) * 32, wj = (wave >> 1) * 32;
    floatx4 acc[2][2] = {};
    for (int64_t r0 = 0; r0 < bytes; r0 += 128) {
        __syncthreads();
        load_any(lp, p + r0, a.ldp, t.rows, bytes - r0);
        load_any(lq, q + r0, a.ldq, cols, bytes - r0);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t block = r0 / 16 + 4 * s + lane / 16;     // this lane's scale block
            MX4::Frag fp[2], fq[2];
            uint32_t ep[2], eq[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int at = (b * 16 + lane % 16) * kAnyPitch + s * 64 + lane / 16 * 16;
                fp[b].v[0] = *reinterpret_cast<const uint4*>(lp + wi * kAnyPitch + at);
                fq[b].v[0] = *reinterpret_cast<const uint4*>(lq + wj * kAnyPitch + at);
                const int i = wi + b * 16 + lane % 16, j = wj + b * 16 + lane % 16;
                ep[b] = i < t.rows && block < kb ? pe[i * a.ldps + block] : 0;
                eq[b] = j < cols && block < kb ? qe[j * a.ldqs + block] : 0;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = MX4::mma<0, 0>(fq[j], fp[i], acc[i][j], eq[j], ep[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = wi + 16 * i + lane % 16, col = wj + 16 * j + 4 * (lane / 16) + e;
                if (row >= t.rows || col >= cols) continue;
                const int64_t at = (t.row0 + row) * a.ldc + j0 + col;
                const float x = acc[i][j][e];
                if (a.out_type == kTypeF32) reinterpret_cast<float*>(a.c)[at] = x;
                else reinterpret_cast<uint16_t*>(a.c)[at] = to_bits16(x, a.out_type);
            }
}

hipError_t launch_any(const MxArgs& a, hipStream_t st)
{
    const uint32_t grid = grid_of(row_tiles(a, kAnyTile) * ((a.J + kAnyTile - 1) / kAnyTile), 256);
    if (!grid) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(mx_any_layout_kernel, dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx(const MxArgs& a, int variant, hipStream_t st)
{
    (void)variant;
    return launch_any(a, st);
}

}  // namespace agg
