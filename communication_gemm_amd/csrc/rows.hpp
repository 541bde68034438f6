// rows.hpp -- eight neighbouring elements of a row a lane: loads and stores of
// 16-bit and float32 rows, of E4M3 codes, and sums and maxima over lanes.
#pragma once

#include "device.hpp"
#include "experts.hpp"
#include "mfma.hpp"

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

// Rounds to kType's bits (in the low half for 16-bit types).
template <int kType>
__device__ __forceinline__ uint32_t narrow_bits(float x)
{
    if constexpr (kType == kTypeF32) return __builtin_bit_cast(uint32_t, x);
    else return to_bits16(x, kType);
}

// Eight neighbouring elements of a row, rounded to kType.  kWide: as load8.
template <int kType, bool kWide>
__device__ __forceinline__ void store_row8(char* row, int64_t col, int64_t k, const float (&v)[8])
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    char* at = row + col * kElt;
    if constexpr (kWide) {
        if (col >= k) return;
        uint32_t w[2 * kElt];
#pragma unroll
        for (int e = 0; e < 2 * kElt; ++e)
            w[e] = kElt == 4 ? narrow_bits<kType>(v[e])
                             : narrow_bits<kType>(v[2 * e % 8]) | narrow_bits<kType>(v[(2 * e + 1) % 8]) << 16;
#pragma unroll
        for (int h = 0; h < kElt / 2; ++h)
            reinterpret_cast<uint4*>(at)[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < k) {
                if constexpr (kElt == 4) reinterpret_cast<uint32_t*>(at)[e] = narrow_bits<kType>(v[e]);
                else reinterpret_cast<uint16_t*>(at)[e] = (uint16_t)narrow_bits<kType>(v[e]);
            }
    }
}

// The sum over a wave, in every lane; the order depends on nothing.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

}  // namespace

}  // namespace agg
