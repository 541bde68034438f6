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

// Eight elements as they lie in memory, 16-byte loads: to be fetched ahead at
// half the registers of their values.
template <int kType>
struct Raw8 {
    uint32_t w[kType == kTypeF32 ? 8 : 4];

    __device__ __forceinline__ void load(const char* row, int64_t col, int64_t k)
    {
        constexpr int kElt = kType == kTypeF32 ? 4 : 2;
#pragma unroll
        for (int e = 0; e < 2 * kElt; ++e) w[e] = 0;
        if (col >= k) return;
#pragma unroll
        for (int h = 0; h < kElt / 2; ++h) {
            const uint4 u = reinterpret_cast<const uint4*>(row + col * kElt)[h];
            w[4 * h] = u.x; w[4 * h + 1] = u.y; w[4 * h + 2] = u.z; w[4 * h + 3] = u.w;
        }
    }

    __device__ __forceinline__ float operator[](int e) const
    {
        if constexpr (kType == kTypeF32) return widen<kType>(w[e]);
        else return widen<kType>(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu);
    }
};

// Another lane's value, by the data-parallel-primitive control `c` (the lanes
// it names all exist).
template <int c>
__device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, c, 0xf, 0xf, false);
}

// The maximum over each four, and over each 16 neighbouring lanes, in all of
// them: lane swaps and rotations of 8, 4, 2 and 1 within 16.
__device__ __forceinline__ uint32_t max4(uint32_t m)
{
    m = max(m, from_lane<0xb1>(m));     // quad_perm [1, 0, 3, 2]
    return max(m, from_lane<0x4e>(m));  // [2, 3, 0, 1]
}

__device__ __forceinline__ uint32_t max16(uint32_t m)
{
    m = max(m, from_lane<0x128>(m));
    m = max(m, from_lane<0x124>(m));
    m = max(m, from_lane<0x122>(m));
    return max(m, from_lane<0x121>(m));
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

// The sum over a wave, in every lane: rotations within 16 lanes, then the four
// sixteens, always in the same order.
__device__ __forceinline__ float wave_sum(float v)
{
    const auto plus = [](float a, uint32_t b) { return a + __builtin_bit_cast(float, b); };
    v = plus(v, from_lane<0x128>(__builtin_bit_cast(uint32_t, v)));
    v = plus(v, from_lane<0x124>(__builtin_bit_cast(uint32_t, v)));
    v = plus(v, from_lane<0x122>(__builtin_bit_cast(uint32_t, v)));
    v = plus(v, from_lane<0x121>(__builtin_bit_cast(uint32_t, v)));
    float s[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
        s[g] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * g));
    return (s[0] + s[1]) + (s[2] + s[3]);
}

}  // namespace

}  // namespace agg
