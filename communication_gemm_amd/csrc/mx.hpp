// mx.hpp -- the matrix instruction of the microscaled 4-bit products.
#pragma once

#include "device.hpp"
#include "layers.hpp"
#include "mfma.hpp"

namespace agg {

namespace {

// E2M1 codes with an E8M0 scale for each 32 of r, 16 x 16 blocks, 128 r an
// instruction: lane l holds the 32 values (16 bytes) number l / 16 of row l %
// 16, one scale block, whose scale is byte kB of the lane's scale operand.  The
// operands are moved as rows of 16-bit units of four values: a step of 32
// units is one instruction.  can(t): outputs of type t; every product of two
// E2M1 values is a multiple of 1/4 below 64, and the instruction adds eight
// neighbouring ones without loss, so float32 outputs need no other form.
struct MX4 {
    static constexpr int kElt = 2, kStep = 32, kFrag = 1;
    static constexpr bool can(int t) { return t == kTypeF16 || t == kTypeBF16 || t == kTypeF32; }
    struct Frag { uint4 v[1]; };

    __device__ __forceinline__ static intx8 wide(const uint4& v)
    {
        return {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
    }

    template <int kQB, int kPB>
    __device__ __forceinline__ static floatx4 mma(const Frag& q, const Frag& p, floatx4 c, uint32_t qs,
                                                  uint32_t ps)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(q.v[0]), wide(p.v[0]), c, 4, 4, kQB,
                                                                (int)qs, kPB, (int)ps);
    }
};

}  // namespace

}  // namespace agg
