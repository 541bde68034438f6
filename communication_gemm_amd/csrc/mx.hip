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

// ---- tiles ---------------------------------------------------------------

template <class E, int BJ>
__device__ __forceinline__ void mx_tile(const MxArgs& a, const TileRef& t, char* ring)
{
    const int64_t j0 = (int64_t)t.j * BJ;
    const int cols = uniform((int)(a.J - j0));
    // rows as 16-bit units of four values
    const typename E::Src s{a.p + t.row0 * a.ldp, a.q + t.group * a.q_stride + j0 * a.ldq, a.ldp / 2, a.ldq / 2,
                            a.R / 4, t.rows, cols < BJ ? cols : BJ};
    const typename E::Scales sc{a.pe + t.row0 * a.ldps, a.qe + t.group * a.qs_stride + j0 * a.ldqs, a.ldps, a.ldqs,
                                (a.R + kMxBlock - 1) / kMxBlock};
    typename E::Acc acc = {};
    E::run(ring, s, sc, acc);
    const int64_t at = t.row0 * a.ldc + j0;
    const int c = cols < BJ ? cols : BJ;
    if (a.out_type == kTypeF32) E::template store<kTypeF32>(ring, a.c + at * 4, a.ldc, t.rows, c, a.c_pieces, acc);
    else if (a.out_type == kTypeF16) E::template store<kTypeF16>(ring, a.c + at * 2, a.ldc, t.rows, c, a.c_pieces, acc);
    else E::template store<kTypeBF16>(ring, a.c + at * 2, a.ldc, t.rows, c, a.c_pieces, acc);
}

// E: MxTile or MxSmallTile of BI x BJ.
template <class E, int BI, int BJ>
__global__ __launch_bounds__(E::kThreads) void mx_tile_kernel(MxArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char ring[];
    TileRef t;
    if (!find_tile<BI, 4>(a, blockIdx.x, (a.J + BJ - 1) / BJ, t)) return;
    mx_tile<E, BJ>(a, t, ring);
}

template <bool kShift>
__global__ __launch_bounds__(512) void mx_large_kernel(MxArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char ring[];
    const uint32_t nj = ((uint32_t)a.J + 255) / 256;
    HalfTiles h;
    h.init(a, nj, (uint32_t)a.cus);
    const uint32_t p = round_position(blockIdx.x, h.positions(), (uint32_t)a.cus);
    if (p >= h.positions()) return;
    TileRef t;
    bool is_half;
    if (!h.tile(a, nj, p, is_half, t)) return;
    if (is_half) mx_tile<MxLargeTile<128, kShift>, 256>(a, t, ring);
    else mx_tile<MxLargeTile<256, kShift>, 256>(a, t, ring);
}

// ---- few rows ---------------------------------------------------------------
//
// Bound by the weights' bytes: as skinny.hip's kernel for weights with r along
// memory, a workgroup owns 16 kMB rows and a strip of 16 kNB columns, its waves
// walk every kWaves-th slice of 256 r with loads of their own, kU slices ahead,
// and their sums are added in wave order.  A slice's eight scales of a row come
// in one load of the three dwords they lie in; lane group g shifts its own down
// (two dwords where rows start on them: 5 x 7168 x 4096 5.66 us, 5.69 so).

template <int kMB, int kNB, int kU>
struct MxBatch {
    uint4 p[kU][kMB][2], q[kU][kNB][2];
    uint32_t ps[kU][kMB][3], qs[kU][kNB][3];
};

template <int kMB, int kNB, int kWaves, int kU>
__global__ __launch_bounds__(64 * kWaves) void mx_skinny_kernel(MxArgs a)
{
    constexpr int BI = 16 * kMB, BJ = 16 * kNB, kBlocks = kMB * kNB;
    __shared__ __attribute__((aligned(16))) floatx4 lds[kWaves * kBlocks * 64];
    TileRef t;
    if (!find_tile<BI, 1>(a, blockIdx.x, (a.J + BJ - 1) / BJ, t)) return;
    const int j0 = t.j * BJ;
    const int cols = a.J - j0 < BJ ? a.J - j0 : BJ;
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int l = lane & 15, g = lane >> 4;
    const uint32_t r_bytes = (uint32_t)a.R / 2;
    const int kb = a.R / kMxBlock;
    const __amdgpu_buffer_rsrc_t rp = scalar_rsrc(a.p + t.row0 * a.ldp, (t.rows - 1) * a.ldp + r_bytes);
    const __amdgpu_buffer_rsrc_t rq =
        scalar_rsrc(a.q + t.group * a.q_stride + j0 * a.ldq, (cols - 1) * a.ldq + r_bytes);
    const uint8_t* pe = a.pe + t.row0 * a.ldps;
    const uint8_t* qe = a.qe + t.group * a.qs_stride + j0 * a.ldqs;
    const __amdgpu_buffer_rsrc_t rps = scale_rsrc<true>(pe, t.rows, a.ldps, kb);
    const __amdgpu_buffer_rsrc_t rqs = scale_rsrc<true>(qe, cols, a.ldqs, kb);
    // of this lane's rows (16 apart the same), and where they start
    const uint32_t p_at = (uint32_t)(l * a.ldps) + skip_of<true>(pe), q_at = (uint32_t)(l * a.ldqs) + skip_of<true>(qe);
    const int nk = (int)((r_bytes + 127) / 128);

    typedef MxBatch<kMB, kNB, kU> B;
    auto load_scales = [&](__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t (&v)[3]) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b96(r, at & ~3u, 0, 0);
        v[0] = x[0];
        v[1] = x[1];
        v[2] = x[2];
    };
    auto load = [&](B& b, int first) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int s = first + u * kWaves;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t byte = (uint32_t)s * 128u + (uint32_t)(h * 64 + g * 16);
                const bool in = byte < r_bytes;
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    b.q[u][j][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                        rq, in ? (uint32_t)((16 * j + l) * a.ldq) + byte : kOutOfRange, 0, 0));
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    b.p[u][i][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                        rp, in ? (uint32_t)((16 * i + l) * a.ldp) + byte : kOutOfRange, 0, 0));
            }
            const bool in = 8 * s < kb;
#pragma unroll
            for (int j = 0; j < kNB; ++j)
                load_scales(rqs, in ? q_at + (uint32_t)(16 * j * a.ldqs + 8 * s) : kOutOfRange, b.qs[u][j]);
#pragma unroll
            for (int i = 0; i < kMB; ++i)
                load_scales(rps, in ? p_at + (uint32_t)(16 * i * a.ldps + 8 * s) : kOutOfRange, b.ps[u][i]);
        }
    };
    floatx4 acc[kMB][kNB] = {};
    auto multiply = [&](const B& b, int first) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // scales behind the row's last are the next row's
                const bool in = 8 * (first + u * kWaves) + 4 * h + g < kb;
                uint32_t ps[kMB], qs[kNB];
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    ps[i] = in ? shifted<true>(b.ps[u][i][h], b.ps[u][i][h + 1], p_at & 3) >> (8 * g) : 0u;
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    qs[j] = in ? shifted<true>(b.qs[u][j][h], b.qs[u][j][h + 1], q_at & 3) >> (8 * g) : 0u;
#pragma unroll
                for (int i = 0; i < kMB; ++i)
#pragma unroll
                    for (int j = 0; j < kNB; ++j)
                        acc[i][j] = MX4::mma<0, 0>({b.q[u][j][h]}, {b.p[u][i][h]}, acc[i][j], qs[j], ps[i]);
            }
    };
    constexpr int kStep = kWaves * kU;
    B b0, b1;
    load(b0, wave);
    for (int s = wave; s < nk; s += 2 * kStep) {
        load(b1, s + kStep);
        multiply(b0, s);
        load(b0, s + 2 * kStep);
        multiply(b1, s + kStep);
    }
#pragma unroll
    for (int j = 0; j < kNB; ++j)
#pragma unroll
        for (int i = 0; i < kMB; ++i) lds[(wave * kBlocks + j * kMB + i) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int u = threadIdx.x; u < kBlocks * 64; u += 64 * kWaves) {
        floatx4 x = lds[u];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const floatx4 y = lds[w * kBlocks * 64 + u];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += y[e];
        }
        const int ul = u & 63, b = u >> 6;
        const int row = b % kMB * 16 + (ul & 15), col = b / kMB * 16 + 4 * (ul >> 4);
        if (row >= t.rows || col >= cols) continue;
        const int64_t at = (t.row0 + row) * a.ldc + j0 + col;
        if (!a.c_pieces) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (col + e >= cols) break;
                if (a.out_type == kTypeF32) reinterpret_cast<float*>(a.c)[at + e] = x[e];
                else reinterpret_cast<uint16_t*>(a.c)[at + e] = to_bits16(x[e], a.out_type);
            }
        } else if (a.out_type == kTypeF32) {      // cols: whole groups of four
            *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(a.c) + at) = x;
        } else {
            const uint32_t lo = to_bits16(x[0], a.out_type) | (uint32_t)to_bits16(x[1], a.out_type) << 16;
            const uint32_t hi = to_bits16(x[2], a.out_type) | (uint32_t)to_bits16(x[3], a.out_type) << 16;
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.c) + at) = make_uint2(lo, hi);
        }
    }
}

// ---- launches -----------------------------------------------------------

hipError_t launch_any(const MxArgs& a, hipStream_t st)
{
    const uint32_t grid = grid_of(row_tiles(a, kAnyTile) * ((a.J + kAnyTile - 1) / kAnyTile), 256);
    if (!grid) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(mx_any_layout_kernel, dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class E, int BI, int BJ>
hipError_t launch_tile(const MxArgs& a, hipStream_t st)
{
    const uint32_t grid = grid_of(row_tiles(a, BI) * ((a.J + BJ - 1) / BJ), E::kThreads);
    if (!grid) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const auto kernel = mx_tile_kernel<E, BI, BJ>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), E::kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(E::kThreads), E::kLds, st, a);
    return hipGetLastError();
}

template <bool kShift>
hipError_t launch_large(const MxArgs& a, hipStream_t st)
{
    constexpr int kLds = MxLargeTile<256, kShift>::kLds;
    // one position a tile, and one more for each tile that is cut in two
    // (at most half a round)
    const int64_t tiles = row_tiles(a, 256) * ((a.J + 255) / 256);
    const int64_t more = tiles < a.cus / 2 ? tiles : a.cus / 2;
    const int64_t wgs = (tiles + more + kXcds - 1) / kXcds * kXcds;
    if (wgs * 512 > 0xffffffffll) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(mx_large_kernel<kShift>), kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mx_large_kernel<kShift>), dim3((uint32_t)wgs), dim3(512), kLds, st, a);
    return hipGetLastError();
}

template <int kMB, int kNB, int kWaves, int kU>
hipError_t launch_skinny(const MxArgs& a, hipStream_t st)
{
    const int64_t nj = (a.J + 16 * kNB - 1) / (16 * kNB);
    const uint32_t grid = grid_of(row_tiles(a, 16 * kMB) * nj, 64 * kWaves);
    if (!grid) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mx_skinny_kernel<kMB, kNB, kWaves, kU>), dim3(grid), dim3(64 * kWaves), 0, st, a);
    return hipGetLastError();
}

template <bool kShift>
hipError_t launch_of(const MxArgs& a, int variant, hipStream_t st)
{
    switch (variant) {
    case kTileLarge: return launch_large<kShift>(a, st);
    case kTile128x128: return launch_tile<MxTile<128, 128, 2, 4, 2, kShift>, 128, 128>(a, st);
    case kTile64x256: return launch_tile<MxTile<64, 256, 2, 4, 2, kShift>, 64, 256>(a, st);
    case kTile64x64: return launch_tile<MxSmallTile<64, 64, 2, 2, 3, 1, kShift>, 64, 64>(a, st);
    case kSplit64x128: return launch_tile<MxSmallTile<64, 128, 2, 2, 3, 2, kShift>, 64, 128>(a, st);
    case kSplit64x64: return launch_tile<MxSmallTile<64, 64, 2, 2, 3, 2, kShift>, 64, 64>(a, st);
    case kSplit32x64: return launch_tile<MxSmallTile<32, 64, 1, 2, 3, 4, kShift>, 32, 64>(a, st);
    case kSplit32x32: return launch_tile<MxSmallTile<32, 32, 1, 1, 2, 8, kShift>, 32, 32>(a, st);
    case kSkinny16: return launch_skinny<1, 1, 4, 2>(a, st);
    case kSkinny32: return launch_skinny<2, 1, 8, 1>(a, st);
    default: return launch_any(a, st);
    }
}

}  // namespace

hipError_t launch_mx(const MxArgs& a, int variant, bool shift, hipStream_t st)
{
    return shift ? launch_of<true>(a, variant, st) : launch_of<false>(a, variant, st);
}

}  // namespace agg
