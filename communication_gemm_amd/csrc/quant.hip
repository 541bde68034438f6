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

namespace agg {

namespace {

constexpr uint32_t kAmaxFloor = 0x0d800000u;   // 2^-100
constexpr float kE4M3Max = 448.f;

template <int kType>
__device__ __forceinline__ float widen(uint32_t bits)
{
    if constexpr (kType == kTypeF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    if constexpr (kType == kTypeBF16) return __builtin_bit_cast(float, bits << 16);
    return __builtin_bit_cast(float, bits);
}

// Eight neighbouring elements.  kWide: 16-byte loads (k, ld and the pointer
// allow them); otherwise one by one, zero past `left`.
template <int kType, bool kWide>
__device__ __forceinline__ void load8(const char* row, int64_t col, int64_t k, float (&v)[8])
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    const char* at = row + col * kElt;
    if constexpr (kWide) {
        uint32_t w[4 * kElt / 2] = {};
        if (col < k) {
#pragma unroll
            for (int h = 0; h < kElt / 2; ++h) {
                const uint4 u = reinterpret_cast<const uint4*>(at)[h];
                w[4 * h] = u.x; w[4 * h + 1] = u.y; w[4 * h + 2] = u.z; w[4 * h + 3] = u.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = kElt == 4 ? widen<kType>(w[e])
                             : widen<kType>(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t b = 0;
            if (col + e < k) {
                if constexpr (kElt == 4) b = reinterpret_cast<const uint32_t*>(at)[e];
                else b = reinterpret_cast<const uint16_t*>(at)[e];
            }
            v[e] = widen<kType>(b);
        }
    }
}

__device__ __forceinline__ uint32_t max_bits(const float (&v)[8])
{
    uint32_t m = 0;   // |x| as bits orders like |x|, with infinities and NaN on top
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}

template <bool kWide>
__device__ __forceinline__ void store8(uint8_t* row, int64_t col, int64_t k, const float (&v)[8],
                                       float inverse)
{
    int w[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inverse, v[4 * h + 1] * inverse, w[h],
                                               false);
        w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inverse, v[4 * h + 3] * inverse, w[h],
                                               true);
    }
    if constexpr (kWide) {
        if (col < k) *reinterpret_cast<uint2*>(row + col) = make_uint2((uint32_t)w[0], (uint32_t)w[1]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < k) row[col + e] = (uint8_t)((uint32_t)w[e / 4] >> (8 * (e % 4)));
    }
}

__device__ __forceinline__ uint32_t max16(uint32_t m)
{
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    return m;
}

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
