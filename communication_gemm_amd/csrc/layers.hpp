// layers.hpp -- arguments and launchers of what stands around the expert
// products: sorting tokens by expert and back (route.hip), the norm
// (norm.hip) and microscaled 4-bit values (mxquant.hip, mx.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "experts.hpp"

namespace agg {

constexpr int kMaxExperts = 4096;   // of a sort: its counts are held in LDS
constexpr int kMxBlock = 32;        // values that one E8M0 scale covers

// ---- route ----------------------------------------------------------------

struct SortArgs {
    const void* ids;         // [tokens, top] of 4 or 8 bytes
    int64_t ld;
    int32_t* offsets;
    int32_t* place;          // [tokens * top]
    int32_t* counts;         // sorts of more than one pass: [blocks, experts]
    int n, top, experts;     // n = tokens * top
    int chunk;               // assignments a workgroup places
};

// Assignments up to which every workgroup counts all of them itself (a pass over
// 1024 of them is 0.25 us; a launch that counts them once 1.5 to 2), and the
// workgroups of a sort and their part: a multiple of 1024, or, of four waves, 256 (32
// tokens, top 8 of 128: 3.4 us, 4.8 with stretches of 256).
constexpr int kSortRecount = 8192;
inline int sort_chunk(int64_t n)
{
    if (n <= 256) return 256;
    const int64_t per = n <= kSortRecount ? 1024 : (n + 255) / 256;
    return (int)((per + 1023) / 1024 * 1024);
}
inline int sort_blocks(int64_t n) { return n ? (int)((n + sort_chunk(n) - 1) / sort_chunk(n)) : 1; }

struct DispatchArgs {
    const char* x;
    char* xs;
    const int32_t* place;
    int64_t ldx, ldxs;       // bytes
    int64_t row_bytes;
    int64_t tokens;
    int top, rows;           // rows of xs
};

struct CombineArgs {
    const char* h;
    const int32_t* place;
    const float* w;          // or nullptr: ones
    char* y;                 // combine: out; gradient: dy
    char* dh;                // gradient: or nullptr
    float* dw;               // gradient: or nullptr
    int64_t ldh, ldw, ldy, lddh, lddw;
    int64_t tokens, k;
    int top, rows;           // rows of h (and dh)
};

hipError_t launch_sort(const SortArgs& a, bool wide_ids, hipStream_t st);
hipError_t launch_dispatch(const DispatchArgs& a, int unit, hipStream_t st);
hipError_t launch_combine(const CombineArgs& a, int type, int out_type, bool wide, hipStream_t st);
hipError_t launch_combine_grad(const CombineArgs& a, int type, bool wide, hipStream_t st);

// ---- norm -----------------------------------------------------------------

struct NormArgs {
    const char* x;
    const char* res;         // or nullptr
    const char* weight;      // or nullptr: ones
    char* h;                 // or nullptr
    char* y;                 // or nullptr
    uint8_t* q;              // or nullptr
    float* scale;
    float* rstd;             // or nullptr
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    int64_t rows, k;
    float eps;
};

struct NormGradArgs {
    const char* dy;
    const char* h;
    const char* weight;      // or nullptr: ones
    const float* rstd;
    const char* dh;          // or nullptr
    char* dx;
    char* dw;                // or nullptr
    float* partial;          // [parts, k]
    int64_t lddy, ldh, lddh, lddx;
    int64_t rows, k;
    int parts;
    int dw_type;
};

// Workgroups of a gradient, each with a part of the weight's.
inline int norm_grad_parts(int64_t rows) { return (int)(rows < 512 ? rows : 512); }

hipError_t launch_norm(const NormArgs& a, int type, bool wide, hipStream_t st);
hipError_t launch_norm_grad(const NormGradArgs& a, int type, bool wide, hipStream_t st);

// ---- microscaled 4-bit values ------------------------------------------------

struct MxQuantArgs {
    const char* x;           // dequantiser: y
    uint8_t* q;              // rows of k / 2 bytes
    uint8_t* scale;
    int64_t rows, k;
    int64_t ldx, ldq, lds;
};

// A product of 4-bit codes: ProductArgs with rows of bytes (ldp, ldq and q_stride
// in bytes, R in values) and, in place of its scales, E8M0 ones (ldps, ldqs and
// qs_stride in bytes).
struct MxArgs : ProductArgs {
    const uint8_t* pe;       // of a row and 32 of k
    const uint8_t* qe;
    bool c_pieces;           // c's rows are whole pieces of 16 bytes
};

hipError_t launch_mx_quant(const MxQuantArgs& a, int type, bool wide, hipStream_t st);
hipError_t launch_mx_dequant(const MxQuantArgs& a, int type, bool wide, hipStream_t st);
// A 4-bit product's kernel: a Variant, or tiles whose groups of waves share r:
enum MxSplit : int {
    kSplit32x32 = 7,     // eight groups of one wave
    kSplit32x64 = 8,     // four of two
    kSplit64x64 = 9,     // two of four
    kSplit64x128 = 10,   // two of four
};

// shift: rows of scales do not all start on dwords.
hipError_t launch_mx(const MxArgs& a, int variant, bool shift, hipStream_t st);

}  // namespace agg
