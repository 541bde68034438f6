// mfma.hpp -- the matrix instructions of the expert products.
#pragma once

#include "device.hpp"
#include "experts.hpp"

namespace agg {

namespace {

// 16 x 16 blocks.  Lane l holds row (column) l % 16 of an operand and, of
// the kStep r that one instruction sums over, the kFrag * 16 bytes number
// l / 16.  The first operand is Q (its rows are the output's columns), the
// second P, so accumulator e of lane l is output row l % 16, column
// 4 (l / 16) + e: four neighbouring columns of one row, and for fp8 one
// row scale for all four.

struct F16 {
    static constexpr int kElt = 2, kStep = 32, kFrag = 1;
    struct Frag { uint4 v[1]; };
    __device__ static floatx4 mma(const Frag& q, const Frag& p, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, q.v[0]),
                                                      __builtin_bit_cast(half8, p.v[0]), c, 0, 0, 0);
    }
};

struct BF16 : F16 {
    __device__ static floatx4 mma(const Frag& q, const Frag& p, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, q.v[0]),
                                                       __builtin_bit_cast(bf16x8, p.v[0]), c, 0, 0,
                                                       0);
    }
};

// One instruction sums a whole scale block of 128 r; format code 0 is E4M3
// and zero scale operands select the unscaled form.
struct FP8 {
    static constexpr int kElt = 1, kStep = 128, kFrag = 2;
    struct Frag { uint4 v[2]; };
    __device__ static floatx4 mma(const Frag& q, const Frag& p, floatx4 c)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            __builtin_bit_cast(intx8, q), __builtin_bit_cast(intx8, p), c, 0, 0, 0, 0, 0, 0);
    }
};

__device__ __forceinline__ uint16_t to_bits16(float x, int type)
{
    if (type == kTypeF16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

}  // namespace

}  // namespace agg
