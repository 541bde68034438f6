// experts.hpp -- arguments and launchers of the expert products (rows
// grouped by expert, 16-bit and block-scaled fp8) and of the quantiser.
//
// Every product is D[i, j] = sum_r P[i, r] Q[j, r] for one group:
//   grouped   i = row of the group, j = output column, r = k
//   wgrad     i = column of x, j = column of dy, r = row of the group
// An operand is "r-contiguous" (r runs along memory) or "r-strided" (its
// i or j runs along memory and r is the row index).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace agg {

// Element types, numbered as ag_gemm_plan's kinds (and F32 behind them).
enum { kTypeF16 = 0, kTypeBF16 = 2, kTypeFP8 = 3, kTypeF32 = 4 };

constexpr int kScaleBlock = 128;   // k (and rows of b) one fp8 scale covers

struct ProductArgs {
    const char* p;             // x, a
    const char* q;             // w, b; dy
    char* c;                   // y; dw
    const float* ps;           // fp8: scale of a row and k block
    const float* qs;           // fp8: scale of a 128 x 128 block of b
    const int32_t* offsets;    // [groups + 1], or nullptr: one group of all rows
    int rows;                  // rows of x (and of y, dy): less than 2^31 - 256
    int groups;
    int64_t ldp, ldq, ldc;     // elements from one row to the next
    int64_t q_stride;          // elements from one group's weights to the next
    int64_t c_stride;          // wgrad: from one group's gradient to the next
    int64_t ldps, ldqs, qs_stride;
    int I, J, R;               // grouped: I unused; wgrad: R unused
    int out_type;
    int cus;                   // of the device, a multiple of 8
};

struct QuantArgs {
    const char* x;
    uint8_t* q;
    float* scale;
    int64_t rows, k;
    int64_t ldx, ldq, lds;
};

// Which kernel a call runs (see pick_* in experts_api.cpp).
enum Variant {
    kAnyLayout = 0,   // 64 x 64 tiles, element loads: every stride and alignment
    kTileLarge = 1,   // 256 x 256 and 128 x 256 tiles, eight waves (this and those
                      // below: whole 16-byte pieces)
    kTile128x128 = 2, // eight waves, two workgroups a CU (fp8: one)
    kTile64x256 = 3,  // eight waves
    kTile64x64 = 4,   // four waves, a deeper ring, two workgroups a CU
    kSkinny16 = 5,    // 16 rows, r split over eight waves
    kSkinny32 = 6,    // 32 rows
};

// type: element type of P and Q; q_strided: Q is r-strided (P is not).
hipError_t launch_grouped(const ProductArgs& a, int type, bool q_strided, int variant,
                          hipStream_t st);
hipError_t launch_skinny(const ProductArgs& a, int type, bool q_strided, int variant, hipStream_t st);
hipError_t launch_wgrad(const ProductArgs& a, int type, int variant, hipStream_t st);
hipError_t launch_quant(const QuantArgs& a, int type, int block_rows, bool wide, hipStream_t st);

}  // namespace agg
