// quant.hip -- 16-bit or float32 rows to E4M3 codes with a float32 scale for
// each 1 x 128 block (activations) or 128 x 128 block (weights):
//
//   amax  = max |x| over the block, at least 2^-100
//   scale = amax / 448                      (448: the largest E4M3 value)
//   q     = E4M3(x * (448 / amax))          (round to nearest, ties to even)
//
// The floor keeps 448 / amax finite: a block of zeros gets zero codes and a
// tiny scale.  A block that holds an infinity or a NaN gets a scale that is
// not finite, so whatever is computed from it is NaN and not a plausible
// number.  HBM-bound: each element is read once and its byte written once,
// 16 bytes in and 8 out a lane; 8192 x 7168 bf16 takes 33.2 us, 5.4 TB/s (a
// large copy reaches 5.1).
#include "device.hpp"
#include "experts.hpp"
#include "rows.hpp"

namespace agg {

namespace {

// 1 x 128 blocks: 16 lanes of eight elements a block, four blocks a wave.
template <int kType, bool kWide>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    const int64_t kb = (a.k + kScaleBlock - 1) / kScaleBlock;
    const int64_t blocks = a.rows * kb;
    const int lane = threadIdx.x % 16;
    const int64_t step = (int64_t)gridDim.x * 16;
    for (int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; b < blocks; b += step) {
        const int64_t row = b / kb, j = b % kb;
        const int64_t col = j * kScaleBlock + lane * 8;
        float v[8];
        load8<kType, kWide>(a.x + row * a.ldx * kElt, col, a.k, v);
        uint32_t m = max16(max_bits(v));
        m = m > kAmaxFloor ? m : kAmaxFloor;
        const float amax = __builtin_bit_cast(float, m);
        store8<kWide>(a.q + row * a.ldq, col, a.k, v, kE4M3Max / amax);
        if (lane == 0) a.scale[row * a.lds + j] = amax / kE4M3Max;
    }
}

// 128 x 128 blocks: one workgroup a block, 16 rows at a time, the block
// kept in registers between the two passes.
template <int kType, bool kWide>
__global__ __launch_bounds__(256) void quant_block_kernel(QuantArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    __shared__ uint32_t top[4];
    const int64_t kb = (a.k + kScaleBlock - 1) / kScaleBlock;
    const int64_t i = blockIdx.x / kb, j = blockIdx.x % kb;
    const int64_t col = j * kScaleBlock + threadIdx.x % 16 * 8;
    const int64_t row0 = i * kScaleBlock + threadIdx.x / 16;
    float v[8][8];
    uint32_t m = kAmaxFloor;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t row = row0 + 16 * u;
        load8<kType, kWide>(a.x + row * a.ldx * kElt, col, row < a.rows ? a.k : 0, v[u]);
        const uint32_t b = max_bits(v[u]);
        m = b > m ? b : m;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if (threadIdx.x % 64 == 0) top[threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = top[w] > m ? top[w] : m;
    const float amax = __builtin_bit_cast(float, m);
    const float inverse = kE4M3Max / amax;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t row = row0 + 16 * u;
        store8<kWide>(a.q + row * a.ldq, col, row < a.rows ? a.k : 0, v[u], inverse);
    }
    if (threadIdx.x == 0) a.scale[i * a.lds + j] = amax / kE4M3Max;
}

template <int kType, bool kWide>
hipError_t launch(const QuantArgs& a, int block_rows, hipStream_t st)
{
    const int64_t kb = (a.k + kScaleBlock - 1) / kScaleBlock;
    if (block_rows == 1) {
        const int64_t wgs = (a.rows * kb + 15) / 16;
        const uint32_t grid = (uint32_t)(wgs < 8192 ? wgs : 8192);
        hipLaunchKernelGGL((quant_rows_kernel<kType, kWide>), dim3(grid), dim3(256), 0, st, a);
    } else {
        const int64_t wgs = (a.rows + kScaleBlock - 1) / kScaleBlock * kb;
        if (wgs * 256 > 0xffffffffll) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((quant_block_kernel<kType, kWide>), dim3((uint32_t)wgs), dim3(256), 0,
                           st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a, int type, int block_rows, bool wide, hipStream_t st)
{
    if (type == kTypeF16)
        return wide ? launch<kTypeF16, true>(a, block_rows, st) : launch<kTypeF16, false>(a, block_rows, st);
    if (type == kTypeBF16)
        return wide ? launch<kTypeBF16, true>(a, block_rows, st) : launch<kTypeBF16, false>(a, block_rows, st);
    return wide ? launch<kTypeF32, true>(a, block_rows, st) : launch<kTypeF32, false>(a, block_rows, st);
}

}  // namespace agg
