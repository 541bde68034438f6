// mxquant.hip -- 16-bit or float32 rows to microscaled 4-bit values, and back:
//
//   amax  = max |x| over 32 columns
//   scale = 2^(floor(log2(amax)) - 2), as its E8M0 code (exponent + 127, at
//           least 0; 255, NaN, where a value is not finite)
//   q     = E2M1(x / scale)      (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives; to
//                                 nearest, ties to even, 6 and above to 6)
//
// E2M1's largest power of two is 4, so x / scale is below 8.  Division by a
// power of two and the values themselves are exact in float32: the codes do
// not depend on how they are computed.  Two codes a byte, the even column in
// its low half.  HBM-bound.
#include "device.hpp"
#include "layers.hpp"
#include "rows.hpp"

namespace agg {

namespace {

// The value of an E8M0 code (2^-127 is a subnormal float32).
__device__ __forceinline__ float e8m0(uint32_t code)
{
    const uint32_t b = code == 0 ? 0x00400000u : code == 255 ? 0x7fc00000u : code << 23;
    return __builtin_bit_cast(float, b);
}

// 4 lanes of eight columns a block.
template <int kType, bool kWide>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxQuantArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    const int64_t kb = (a.k + kMxBlock - 1) / kMxBlock;
    const int64_t blocks = a.rows * kb;
    const int lane = threadIdx.x % 4;
    const int64_t step = (int64_t)gridDim.x * 64;
    for (int64_t b = (int64_t)blockIdx.x * 64 + threadIdx.x / 4; b < blocks; b += step) {
        const int64_t row = b / kb, j = b % kb;
        const int64_t col = j * kMxBlock + lane * 8;
        float v[8];
        load8<kType, kWide>(a.x + row * a.ldx * kElt, col, a.k, v);
        const uint32_t m = max4(max_bits(v));
        const int top = (int)(m >> 23);                // 255: not finite
        const int code = top == 255 ? 255 : top > 2 ? top - 2 : 0;     // 0 .. 252, or 255
        uint32_t w = 0;
        if (code != 255) {     // a block that is not finite gets zero codes
            const float inverse = __builtin_bit_cast(float, (uint32_t)(254 - code) << 23);   // 2^(127 - code)
            w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32((int)w, v[0] * inverse, v[1] * inverse, 1.f, 0);
            w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32((int)w, v[2] * inverse, v[3] * inverse, 1.f, 1);
            w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32((int)w, v[4] * inverse, v[5] * inverse, 1.f, 2);
            w = (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32((int)w, v[6] * inverse, v[7] * inverse, 1.f, 3);
        }
        uint8_t* out = a.q + row * a.ldq + col / 2;
        if constexpr (kWide) {
            if (col < a.k) *reinterpret_cast<uint32_t*>(out) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + 2 * e < a.k) out[e] = (uint8_t)(w >> 8 * e);
        }
        if (lane == 0) a.scale[row * a.lds + j] = (uint8_t)code;
    }
}

// Eight columns a lane.
template <int kType, bool kWide>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxQuantArgs a)
{
    constexpr int kElt = kType == kTypeF32 ? 4 : 2;
    const int64_t per = (a.k + 7) / 8;
    const int64_t all = a.rows * per, step = (int64_t)gridDim.x * 256;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += step) {
        const int64_t row = u / per, col = u % per * 8;
        const uint8_t* in = a.q + row * a.ldq + col / 2;
        uint32_t w = 0;
        if constexpr (kWide) {
            w = *reinterpret_cast<const uint32_t*>(in);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + 2 * e < a.k) w |= (uint32_t)in[e] << 8 * e;
        }
        const float s = e8m0(a.scale[row * a.lds + col / kMxBlock]);
        float v[8];
        const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0);
        const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
        const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2);
        const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
        v[0] = v0[0] * s; v[1] = v0[1] * s; v[2] = v1[0] * s; v[3] = v1[1] * s;
        v[4] = v2[0] * s; v[5] = v2[1] * s; v[6] = v3[0] * s; v[7] = v3[1] * s;
        store_row8<kType, kWide>(const_cast<char*>(a.x) + row * a.ldx * kElt, col, a.k, v);
    }
}

template <int kType, bool kWide>
hipError_t launch_quant_of(const MxQuantArgs& a, hipStream_t st)
{
    const int64_t wgs = (a.rows * ((a.k + kMxBlock - 1) / kMxBlock) + 63) / 64;
    hipLaunchKernelGGL((mx_quant_kernel<kType, kWide>), dim3((uint32_t)(wgs < 8192 ? wgs : 8192)), dim3(256), 0,
                       st, a);
    return hipGetLastError();
}

template <int kType, bool kWide>
hipError_t launch_dequant_of(const MxQuantArgs& a, hipStream_t st)
{
    const int64_t wgs = (a.rows * ((a.k + 7) / 8) + 255) / 256;
    hipLaunchKernelGGL((mx_dequant_kernel<kType, kWide>), dim3((uint32_t)(wgs < 8192 ? wgs : 8192)), dim3(256), 0,
                       st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quant(const MxQuantArgs& a, int type, bool wide, hipStream_t st)
{
    if (type == kTypeF16)
        return wide ? launch_quant_of<kTypeF16, true>(a, st) : launch_quant_of<kTypeF16, false>(a, st);
    if (type == kTypeBF16)
        return wide ? launch_quant_of<kTypeBF16, true>(a, st) : launch_quant_of<kTypeBF16, false>(a, st);
    return wide ? launch_quant_of<kTypeF32, true>(a, st) : launch_quant_of<kTypeF32, false>(a, st);
}

hipError_t launch_mx_dequant(const MxQuantArgs& a, int type, bool wide, hipStream_t st)
{
    if (type == kTypeF16)
        return wide ? launch_dequant_of<kTypeF16, true>(a, st) : launch_dequant_of<kTypeF16, false>(a, st);
    if (type == kTypeBF16)
        return wide ? launch_dequant_of<kTypeBF16, true>(a, st) : launch_dequant_of<kTypeBF16, false>(a, st);
    return wide ? launch_dequant_of<kTypeF32, true>(a, st) : launch_dequant_of<kTypeF32, false>(a, st);
}

}  // namespace agg
