// experts.hip -- products of rows grouped by expert: 16-bit forward and
// input gradient (y = x_e W_e, x_e W_e^T), weight gradient (x_e^T dy_e), and
// the E4M3 product with a float32 scale for each 128 of k.
#include <atomic>
#include <type_traits>

#include "device.hpp"
#include "experts.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "mfma.hpp"
#include "tile.hpp"

namespace agg {

namespace {

// ---- every layout -------------------------------------------------------
//
// 64 x 64 tiles, four waves of 32 x 32, one 128-byte slice of r at a time,
// elements loaded one by one with both edges checked: right for any
// stride, alignment and size.  The kernel behind calls whose rows do not
// start on 16-byte boundaries; bound by its element loads.

constexpr int kAnyTile = 64;
constexpr int kAnyPitch = 128 + 16;   // bytes of an LDS row: 16-byte reads of 16
                                      // rows fall on different banks

// A 64 x kR tile of one operand into LDS rows of r.  `strided`: r is the
// row index of memory.
template <int kElt, int kR>
__device__ __forceinline__ void load_any(char* lds, const char* src, bool strided, int64_t ld,
                                         int rows, int r_left)
{
    typedef std::conditional_t<kElt == 2, uint16_t, uint8_t> E;
    const E* s = reinterpret_cast<const E*>(src);
#pragma unroll 4
    for (int u = threadIdx.x; u < kAnyTile * kR; u += 256) {
        const int i = strided ? u % kAnyTile : u / kR;
        const int r = strided ? u / kAnyTile : u % kR;
        E v = 0;
        if (i < rows && r < r_left) v = s[strided ? r * ld + i : i * ld + r];
        *reinterpret_cast<E*>(lds + i * kAnyPitch + r * kElt) = v;
    }
}

template <class T, bool kWgrad>
__global__ __launch_bounds__(256) void any_layout_kernel(ProductArgs a, bool q_strided)
{
    constexpr int kR = 128 / T::kElt;
    __shared__ __attribute__((aligned(16))) char lds[2 * kAnyTile * kAnyPitch];
    char* lp = lds;
    char* lq = lds + kAnyTile * kAnyPitch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nj = (a.J + kAnyTile - 1) / kAnyTile;
    const char* p;
    const char* q;
    int64_t r_all, out0;
    int rows, j0, group;
    if constexpr (kWgrad) {
        const int ni = (a.I + kAnyTile - 1) / kAnyTile;
        const int64_t per = (int64_t)ni * nj;
        group = (int)(blockIdx.x / per);
        const int in = (int)(blockIdx.x % per);
        const int i0 = in / nj * kAnyTile;
        j0 = in % nj * kAnyTile;
        int lo, hi;
        group_rows(a, group, lo, hi);
        r_all = hi - lo;
        rows = a.I - i0 < kAnyTile ? a.I - i0 : kAnyTile;
        p = a.p + (lo * a.ldp + i0) * T::kElt;
        q = a.q + (lo * a.ldq + j0) * T::kElt;
        out0 = group * a.c_stride + i0 * a.ldc;
    } else {
        TileRef t;
        if (!find_tile<kAnyTile, 4>(a, blockIdx.x, nj, t)) return;
        group = t.group;
        rows = t.rows;
        j0 = t.j * kAnyTile;
        r_all = a.R;
        p = a.p + t.row0 * a.ldp * T::kElt;
        q = a.q + (group * a.q_stride + (q_strided ? j0 : j0 * a.ldq)) * T::kElt;
        out0 = t.row0 * a.ldc;
        if constexpr (T::kElt == 1) {
            a.ps += t.row0 * a.ldps;
            a.qs += group * a.qs_stride + j0 / kScaleBlock * a.ldqs;
        }
    }
    const int cols = a.J - j0 < kAnyTile ? a.J - j0 : kAnyTile;
    const int wi = (wave & 1) * 32, wj = (wave >> 1) * 32;
    const int out = output_of<T>(a.out_type);
    floatx4 acc[2][2] = {};
    for (int64_t r0 = 0; r0 < r_all; r0 += kR) {
        const int r_left = r_all - r0 < kR ? (int)(r_all - r0) : kR;
        __syncthreads();
        load_any<T::kElt, kR>(lp, p + r0 * (kWgrad ? a.ldp : 1) * T::kElt, kWgrad, a.ldp, rows,
                              r_left);
        load_any<T::kElt, kR>(lq, q + r0 * (kWgrad || q_strided ? a.ldq : 1) * T::kElt,
                              kWgrad || q_strided, a.ldq, cols, r_left);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kR / T::kStep; ++s) {
            typename T::Frag fp[2], fq[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < T::kFrag; ++h) {
                    const int at = (b * 16 + lane % 16) * kAnyPitch +
                                   (s * 4 + lane / 16) * 16 * T::kFrag + h * 16;
                    fp[b].v[h] = *reinterpret_cast<const uint4*>(lp + wi * kAnyPitch + at);
                    fq[b].v[h] = *reinterpret_cast<const uint4*>(lq + wj * kAnyPitch + at);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (T::kElt == 1) {
                    const int row = wi + 16 * i + lane % 16;
                    const int64_t kb = r0 / kScaleBlock;
                    const float scale = row < rows ? a.ps[row * a.ldps + kb] * a.qs[kb] : 0.f;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const floatx4 part = T::mma(fq[j], fp[i], floatx4{});
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] += part[e] * scale;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = T::mma(fq[j], fp[i], acc[i][j]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = wi + 16 * i + lane % 16;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = wj + 16 * j + 4 * (lane / 16) + e;
                if (row < rows && col < cols) {
                    const int64_t at = out0 + row * a.ldc + j0 + col;
                    const float x = acc[i][j][e];
                    if (out == kTypeF32)
                        reinterpret_cast<float*>(a.c)[at] = x;
                    else
                        reinterpret_cast<uint16_t*>(a.c)[at] = to_bits16(x, out);
                }
            }
    }
}

// ---- tiles ---------------------------------------------------------------
//
// See tile.hpp for the engine.  Which tile a call takes is measured in
// experts_api.cpp; the large kernel is bound by the matrix cores and their
// operands' movement, 64 x 256 and 64 x 64 by the weights' bytes (1001 rows
// over 24 experts of 2056 x 1544: 40.5 us, 3.9 TB/s, where 512-byte rows of w
// against 256-byte ones took 49).

template <class E, bool kStream>
__device__ __forceinline__ void store_any(char* ring, const ProductArgs& a, int64_t at, int rows,
                                          int cols, typename E::Acc& acc)
{
    typedef typename E::Type T;
    const int out = output_of<T>(a.out_type);
    if constexpr (T::can(kTypeF32))
        if (out == kTypeF32)
            return E::template store<kTypeF32, kStream>(ring, a.c + at * 4, a.ldc, rows, cols, acc);
    if constexpr (T::can(kTypeF16))
        if (out == kTypeF16)
            return E::template store<kTypeF16, kStream>(ring, a.c + at * 2, a.ldc, rows, cols, acc);
    if constexpr (T::can(kTypeBF16))
        E::template store<kTypeBF16, kStream>(ring, a.c + at * 2, a.ldc, rows, cols, acc);
}

// One tile of a grouped product.
template <class T, class E, int BI, int BJ, int WJ, bool kQS>
__device__ __forceinline__ void grouped_tile(const ProductArgs& a, const TileRef& t, char* ring)
{
    const int64_t j0 = (int64_t)t.j * BJ;
    const int cols = uniform((int)(a.J - j0));
    const typename E::Src s{a.p + t.row0 * a.ldp * T::kElt,
                            a.q + (t.group * a.q_stride + (kQS ? j0 : j0 * a.ldq)) * T::kElt,
                            a.ldp, a.ldq, a.R, t.rows, kQS || cols < BJ ? cols : BJ};
    typename E::Acc acc = {};
    if constexpr (T::kElt == 1) {
        const int64_t jb = (j0 + (threadIdx.x >> 6) % WJ * (BJ / WJ)) / kScaleBlock;
        const int64_t nb = (a.J + kScaleBlock - 1) / kScaleBlock;   // columns past J: any scale
        E::run8(ring, s, {a.ps + t.row0 * a.ldps,
                          a.qs + t.group * a.qs_stride + (jb < nb ? jb : nb - 1) * a.ldqs, a.ldps,
                          (a.R + kScaleBlock - 1) / kScaleBlock, t.rows}, acc);
    } else {
        E::run16(ring, s, acc);
    }
    store_any<E, false>(ring, a, t.row0 * a.ldc + j0, t.rows, cols < BJ ? cols : BJ, acc);
}

template <class T, int BI, int BJ, int WI, int WJ, int NS, bool kQS>
__global__ __launch_bounds__(64 * WI * WJ) void grouped_tile_kernel(ProductArgs a)
{
    typedef Tile<T, BI, BJ, WI, WJ, NS, false, kQS> E;
    extern __shared__ __attribute__((aligned(16))) char ring[];
    TileRef t;
    if (!find_tile<BI, 4>(a, blockIdx.x, (a.J + BJ - 1) / BJ, t)) return;
    grouped_tile<T, E, BI, BJ, WJ, kQS>(a, t, ring);
}

// Whole and half tiles of 256 columns (HalfTiles), one a workgroup: the
// rings take all of a CU's LDS, so a round is one workgroup a CU.
template <class T, bool kQS>
__global__ __launch_bounds__(512) void grouped_large_kernel(ProductArgs a)
{
    // fp8: a wave 128 columns wide has half the row scales to hold
    constexpr int WI = T::kElt == 1 ? 4 : 2, WJ = 8 / WI;
    typedef Tile<T, 256, 256, WI, WJ, 2, false, kQS> Whole;
    typedef Tile<T, 128, 256, 2, 4, 2, false, kQS> Half;
    extern __shared__ __attribute__((aligned(16))) char ring[];
    const uint32_t nj = ((uint32_t)a.J + 255) / 256;
    HalfTiles h;
    h.init(a, nj, (uint32_t)a.cus);
    const uint32_t p = round_position(blockIdx.x, h.positions(), (uint32_t)a.cus);
    if (p >= h.positions()) return;
    TileRef t;
    bool is_half;
    if (!h.tile(a, nj, p, is_half, t)) return;
    if (is_half) grouped_tile<T, Half, 128, 256, 4, kQS>(a, t, ring);
    else grouped_tile<T, Whole, 256, 256, WJ, kQS>(a, t, ring);
}

template <class T, int BI, int BJ, int WI, int WJ, int NS>
__global__ __launch_bounds__(64 * WI * WJ) void wgrad_tile_kernel(ProductArgs a)
{
    typedef Tile<T, BI, BJ, WI, WJ, NS, true, true> E;
    extern __shared__ __attribute__((aligned(16))) char ring[];
    const int ni = (a.I + BI - 1) / BI, nj = (a.J + BJ - 1) / BJ;
    const uint32_t per = (uint32_t)ni * (uint32_t)nj, tiles = (uint32_t)a.groups * per;
    const uint32_t p = round_position(blockIdx.x, tiles, (uint32_t)a.cus * (163840 / E::kLds));
    if (p >= tiles) return;
    const int group = (int)(p / per), in = (int)(p % per);
    // blocks of four tiles along i, column by column
    const int panel = in / (4 * nj), left = ni - 4 * panel, high = left < 4 ? left : 4;
    const int rest = in - 4 * panel * nj;
    const int64_t i0 = (int64_t)(4 * panel + rest % high) * BI, j0 = (int64_t)(rest / high) * BJ;
    int lo, hi;
    group_rows(a, group, lo, hi);
    lo = uniform(lo);
    hi = uniform(hi);
    const int rows = uniform((int)(a.I - i0)), cols = uniform((int)(a.J - j0));
    const typename E::Src s{a.p + ((int64_t)lo * a.ldp + i0) * T::kElt,
                            a.q + ((int64_t)lo * a.ldq + j0) * T::kElt,
                            a.ldp, a.ldq, hi - lo, rows, cols};
    typename E::Acc acc = {};
    E::run16(ring, s, acc);
    // Gradients that the last-level cache (256 MiB) would not hold anyway
    // are stored past it: 268 MB of fp32 282 us against 305; 63 MB of fp16
    // 31 against 23.  (128 x 128 tiles are for fewer than 256 of 256 x 256, 64
    // MiB of fp32 at most.)
    const int64_t at = group * a.c_stride + i0 * a.ldc + j0;
    const int r = rows < BI ? rows : BI, c = cols < BJ ? cols : BJ;
    if constexpr (BI == 256)
        if ((int64_t)a.groups * a.I * a.J * (a.out_type == kTypeF32 ? 4 : 2) > 128ll << 20)
            return store_any<E, true>(ring, a, at, r, c, acc);
    store_any<E, false>(ring, a, at, r, c, acc);
}

// ---- launches -----------------------------------------------------------

template <class T, bool kWgrad>
hipError_t launch_any(const ProductArgs& a, bool q_strided, hipStream_t st)
{
    const int64_t nj = (a.J + kAnyTile - 1) / kAnyTile;
    const int64_t tiles = kWgrad ? a.groups * ((int64_t)(a.I + kAnyTile - 1) / kAnyTile) * nj
                                 : row_tiles(a, kAnyTile) * nj;
    const uint32_t grid = kWgrad ? (tiles * 256 > 0xffffffffll ? 0 : (uint32_t)tiles)
                                 : grid_of(tiles, 256);
    if (!grid) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((any_layout_kernel<T, kWgrad>), dim3(grid), dim3(256), 0, st, a, q_strided);
    return hipGetLastError();
}

template <class T, int BI, int BJ, int WI, int WJ, int NS, bool kQS>
hipError_t launch_grouped_tile(const ProductArgs& a, hipStream_t st)
{
    typedef Tile<T, BI, BJ, WI, WJ, NS, false, kQS> E;
    const uint32_t grid = grid_of(row_tiles(a, BI) * ((a.J + BJ - 1) / BJ), E::kThreads);
    if (!grid) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const auto kernel = grouped_tile_kernel<T, BI, BJ, WI, WJ, NS, kQS>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), E::kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(E::kThreads), E::kLds, st, a);
    return hipGetLastError();
}

template <class T, bool kQS>
hipError_t launch_large(const ProductArgs& a, hipStream_t st)
{
    constexpr int kLds = Tile<T, 256, 256, 2, 4, 2, false, kQS>::kLds;
    // one position a tile, and one more for each tile that is cut in two
    // (at most half a round)
    const int64_t tiles = row_tiles(a, 256) * ((a.J + 255) / 256);
    const int64_t more = tiles < a.cus / 2 ? tiles : a.cus / 2;
    const int64_t wgs = (tiles + more + kXcds - 1) / kXcds * kXcds;
    if (wgs * 512 > 0xffffffffll) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const auto kernel = grouped_large_kernel<T, kQS>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)wgs), dim3(512), kLds, st, a);
    return hipGetLastError();
}

template <class T, int BI, int BJ, int WI, int WJ, int NS>
hipError_t launch_wgrad_tile(const ProductArgs& a, hipStream_t st)
{
    typedef Tile<T, BI, BJ, WI, WJ, NS, true, true> E;
    const int64_t tiles = (int64_t)((a.I + BI - 1) / BI) * ((a.J + BJ - 1) / BJ) * a.groups;
    const uint32_t grid = grid_of(tiles, E::kThreads);
    if (!grid) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const auto kernel = wgrad_tile_kernel<T, BI, BJ, WI, WJ, NS>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), E::kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(E::kThreads), E::kLds, st, a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_grouped16(const ProductArgs& a, bool q_strided, int variant, hipStream_t st)
{
    if (variant == kTileLarge)
        return q_strided ? launch_large<T, true>(a, st) : launch_large<T, false>(a, st);
    if (variant == kTile64x256)
        return q_strided ? launch_grouped_tile<T, 64, 256, 2, 4, 2, true>(a, st)
                         : launch_grouped_tile<T, 64, 256, 2, 4, 2, false>(a, st);
    if (variant == kTile128x128)
        return q_strided ? launch_grouped_tile<T, 128, 128, 2, 4, 2, true>(a, st)
                         : launch_grouped_tile<T, 128, 128, 2, 4, 2, false>(a, st);
    if (variant == kTile64x64)
        return q_strided ? launch_grouped_tile<T, 64, 64, 2, 2, 4, true>(a, st)
                         : launch_grouped_tile<T, 64, 64, 2, 2, 4, false>(a, st);
    return launch_any<T, false>(a, q_strided, st);
}

// Float32 outputs (FP8Exact): 128 x 128 tiles in the large ones' place, on one
// card 312 against 327 us for 8192 x 4096 x 4096, 160 against 196 for 8000 rows
// of 16 groups of 4096 x 2048, 65 against 68 for 3001 of 32 of 2048 x 2816 (on
// another 315 and 167 for the first two).
template <class T>
hipError_t launch_grouped8(const ProductArgs& a, int variant, hipStream_t st)
{
    if constexpr (std::is_same_v<T, FP8>)
        if (variant == kTileLarge) return launch_large<T, false>(a, st);
    if (variant == kTile128x128 || variant == kTileLarge) return launch_grouped_tile<T, 128, 128, 4, 2, 2, false>(a, st);
    if (variant == kTile64x256) return launch_grouped_tile<T, 64, 256, 1, 8, 2, false>(a, st);
    if (variant == kTile64x64) return launch_grouped_tile<T, 64, 64, 2, 2, 4, false>(a, st);
    return launch_any<T, false>(a, false, st);
}

}  // namespace

hipError_t launch_grouped(const ProductArgs& a, int type, bool q_strided, int variant,
                          hipStream_t st)
{
    if (variant == kSkinny16 || variant == kSkinny32)
        return launch_skinny(a, type, q_strided, variant, st);
    if (type == kTypeF16) return launch_grouped16<F16>(a, q_strided, variant, st);
    if (type == kTypeBF16) return launch_grouped16<BF16>(a, q_strided, variant, st);
    return a.out_type == kTypeF32 ? launch_grouped8<FP8Exact>(a, variant, st)
                                  : launch_grouped8<FP8>(a, variant, st);
}

hipError_t launch_wgrad(const ProductArgs& a, int type, int variant, hipStream_t st)
{
    if (variant == kTileLarge)
        return type == kTypeF16 ? launch_wgrad_tile<F16, 256, 256, 2, 4, 2>(a, st)
                                : launch_wgrad_tile<BF16, 256, 256, 2, 4, 2>(a, st);
    if (variant == kTile128x128)
        return type == kTypeF16 ? launch_wgrad_tile<F16, 128, 128, 2, 4, 2>(a, st)
                                : launch_wgrad_tile<BF16, 128, 128, 2, 4, 2>(a, st);
    return type == kTypeF16 ? launch_any<F16, true>(a, true, st)
                            : launch_any<BF16, true>(a, true, st);
}

}  // namespace agg
