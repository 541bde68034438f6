// experts_api.cpp -- the C ABI of the expert products and the quantiser:
// argument checks (before any HIP call) and the choice of kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "aggemm.h"
#include "checks.hpp"
#include "experts.hpp"

namespace agg {
namespace {

// The kernel of a grouped call, from the sizes the host knows: the mean of
// the groups' rows (were as many groups used as can be; groups of random
// sizes need about a quarter more) and the workgroups each tile would give.
// us per call, bf16 with w r-strided / r-contiguous / fp8, E groups of `mean`
// rows on average:
//   many groups of few rows.  E 32, K 4096, N 2048, mean 8 and 48: 64 x 256
//     91 / 120 / 67 and 94 / 124 / 68, large 91 / 123 / 70 and 93 / 126 / 71,
//     64 x 64 135 / 136 / 93 and 138 / 132 / 85; E 24, K 2056, N 1544, mean 42:
//     64 x 256 40, large 47, 64 x 64 57; E 64, K 2048, N 1408, mean 8: 73 / 89 /
//     42, 80 / 97 / 47, 71 / 81 / 45;
//   very few, w r-contiguous.  E 32, K 4096, N 2048, mean 4 and 8: 16 rows 105 /
//     58 and 126 / 63, large 121 / 69 and 125 / 72; but with rows of w of
//     2 KiB (fp8, E 64, K 2048, N 1408, mean 4): 16 rows 60, 64 x 256 41;
//   few groups of few rows.  E 8, K 4096, N 2048, mean 8 and 48: 64 x 64 30 / 33
//     / 18 and 32 / 32 / 18, 64 x 256 51 / 51 / 24 and 53 / 55 / 25, 32 rows 33 /
//     38 / 20 and 50 / 73 / 49;
//   one matrix.  K 7168, N 4096, 1 / 16 / 32 / 64 rows: 16 rows 24 / 25 / 27 / 42,
//     32 rows 23 / 25 / 28 / 30, 64 x 64 40; 256 rows: 64 x 64 42, 128 x 128 61;
//   more rows.  E 8, mean 64 / 96 / 128 / 256 / 512: 128 x 128 43 / 44 / 44 / 76 /
//     99, large 59 / 62 / 60 / 65 / 100, 64 x 64 51 / 46 / 59 / 89 / 148; E 32,
//     N 1408, mean 64 / 128 / 256 / 512: large 45 / 52 / 85 / 108, 128 x 128
//     44 / 74 / 78 / 132.
int pick(const ProductArgs& a, int elt, bool q_strided, bool whole)
{
    if (!whole) return kAnyLayout;
    const int64_t used = a.groups < a.rows ? a.groups : a.rows;
    const int64_t mean = tiles_of(a.rows, used);
    if (mean <= 48 || (used == 1 && mean <= 64)) {
        if (!q_strided && mean <= 8 && (int64_t)a.R * elt >= 4096) return kSkinny16;
        if (used * tiles_of(a.J, 256) >= 128) return kTile64x256;
        if (used * tiles_of(a.J, 64) >= 200 && mean > 8) return kTile64x64;
        if (mean <= 16) return kSkinny16;
        return used == 1 || mean <= 32 ? kSkinny32 : kTile64x64;
    }
    const int64_t rows = used == 1 ? mean : mean + mean / 4;
    if (used * tiles_of(rows, 128) * tiles_of(a.J, 256) >= 160) return kTileLarge;
    const int64_t tiles128 = used * tiles_of(rows, 128) * tiles_of(a.J, 128);
    return tiles128 >= (used == 1 ? 200 : 120) ? kTile128x128 : kTile64x64;
}

// The kernel of a weight gradient: 256 x 256 tiles, or 128 x 128 where those
// would leave CUs idle.  us, 256 / 128: 8 groups of 512 rows, 4096 x 2048:
// 76 / 89; of 1024 x 1024: 20 / 16; 20 groups of 256 rows, 1024 x 1544 (560
// tiles): 39 / 38.
int pick_wgrad(const ProductArgs& a, bool whole)
{
    if (!whole) return kAnyLayout;
    return a.groups * tiles_of(a.I, 256) * tiles_of(a.J, 256) >= a.cus ? kTileLarge : kTile128x128;
}

int run_fp8(const void* a, int64_t lda, const float* as, int64_t ldas, const void* b, int64_t ldb,
            int64_t b_stride, const float* bs, int64_t ldbs, int64_t bs_stride,
            const int32_t* offsets, int64_t groups, void* c, int64_t ldc, int out_type,
            int64_t M, int64_t K, int64_t N, void* stream)
{
    int rc = check_sizes(M, K, N, groups);
    if (rc) return rc;
    if (out_type != kTypeF32 && !is16(out_type)) return AGG_E_INVALID;
    const int64_t kb = (K + kScaleBlock - 1) / kScaleBlock;
    const int64_t nb = (N + kScaleBlock - 1) / kScaleBlock;
    rc = first_error({check_matrix(a, M, K, lda, 1), check_matrix(as, M, kb, ldas, 4),
                      check_matrix(b, N, K, ldb, 1), check_matrix(bs, nb, kb, ldbs, 4),
                      check_matrix(c, M, N, ldc, elt_of(out_type))});
    if (rc) return rc;
    if (b_stride < 0 || bs_stride < 0) return AGG_E_INVALID;
    if (M == 0) return AGG_OK;
    ProductArgs p{};
    p.p = static_cast<const char*>(a);
    p.q = static_cast<const char*>(b);
    p.c = static_cast<char*>(c);
    p.ps = as;
    p.qs = bs;
    p.offsets = offsets;
    p.rows = (int)M;
    p.ldp = lda;
    p.ldq = ldb;
    p.ldc = ldc;
    p.q_stride = b_stride;
    p.ldps = ldas;
    p.ldqs = ldbs;
    p.qs_stride = bs_stride;
    p.groups = (int)groups;
    p.J = (int)N;
    p.R = (int)K;
    p.out_type = out_type;
    rc = device_cus(&p.cus);
    if (rc) return rc;
    const bool whole = pieces(a, lda, 0, K, 1) && pieces(b, ldb, b_stride, K, 1) &&
                       pieces(c, ldc, 0, N, elt_of(out_type));
    return status_of(launch_grouped(p, kTypeFP8, false, pick(p, 1, false, whole),
                                    static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace agg

using namespace agg;

extern "C" {

int ag_gemm_grouped(int type, const void* x, int64_t ldx, const void* w, int64_t ldw,
                    int64_t w_stride, int trans_w, const int32_t* offsets, int n_groups, void* y,
                    int64_t ldy, int out_type, int64_t T, int64_t K, int64_t N, void* stream)
{
    int rc = check_sizes(T, K, N, n_groups);
    if (rc) return rc;
    if (!is16(type) || (out_type != kTypeF32 && out_type != type)) return AGG_E_INVALID;
    if (!offsets || w_stride < 0) return AGG_E_INVALID;
    rc = first_error({check_matrix(x, T, K, ldx, 2),
                      check_matrix(w, 1, trans_w ? K : N, ldw, 2),
                      check_matrix(y, T, N, ldy, elt_of(out_type))});
    if (rc) return rc;
    if (!aligned(offsets, 4)) return AGG_E_UNSUPPORTED;
    if (T == 0) return AGG_OK;
    ProductArgs p{};
    p.p = static_cast<const char*>(x);
    p.q = static_cast<const char*>(w);
    p.c = static_cast<char*>(y);
    p.offsets = offsets;
    p.rows = (int)T;
    p.ldp = ldx;
    p.ldq = ldw;
    p.ldc = ldy;
    p.q_stride = w_stride;
    p.groups = n_groups;
    p.J = (int)N;
    p.R = (int)K;
    p.out_type = out_type;
    rc = device_cus(&p.cus);
    if (rc) return rc;
    const bool whole = pieces(x, ldx, 0, K, 2) && pieces(w, ldw, w_stride, trans_w ? K : N, 2) &&
                       pieces(y, ldy, 0, N, elt_of(out_type));
    return status_of(launch_grouped(p, type, !trans_w, pick(p, 2, !trans_w, whole),
                                    static_cast<hipStream_t>(stream)));
}

int ag_gemm_grouped_wgrad(int type, const void* x, int64_t ldx, const void* dy, int64_t lddy,
                          const int32_t* offsets, int n_groups, void* dw, int64_t lddw,
                          int64_t dw_stride, int out_type, int64_t T, int64_t K, int64_t N,
                          void* stream)
{
    int rc = check_sizes(T, K, N, n_groups);
    if (rc) return rc;
    if (!is16(type) || (out_type != kTypeF32 && out_type != type)) return AGG_E_INVALID;
    if (!offsets) return AGG_E_INVALID;
    rc = first_error({check_matrix(x, T, K, ldx, 2), check_matrix(dy, T, N, lddy, 2),
                      check_matrix(dw, K, N, lddw, elt_of(out_type))});
    if (rc) return rc;
    // groups' gradients may not overlap
    if (n_groups > 1 && dw_stride < (K - 1) * lddw + N) return AGG_E_INVALID;
    if (!aligned(offsets, 4)) return AGG_E_UNSUPPORTED;
    ProductArgs p{};
    p.p = static_cast<const char*>(x);
    p.q = static_cast<const char*>(dy);
    p.c = static_cast<char*>(dw);
    p.offsets = offsets;
    p.rows = (int)T;
    p.ldp = ldx;
    p.ldq = lddy;
    p.ldc = lddw;
    p.c_stride = dw_stride;
    p.groups = n_groups;
    p.I = (int)K;
    p.J = (int)N;
    p.out_type = out_type;
    rc = device_cus(&p.cus);
    if (rc) return rc;
    const bool whole = pieces(x, ldx, 0, K, 2) && pieces(dy, lddy, 0, N, 2) &&
                       pieces(dw, lddw, dw_stride, N, elt_of(out_type));
    return status_of(launch_wgrad(p, type, pick_wgrad(p, whole),
                                  static_cast<hipStream_t>(stream)));
}

int ag_gemm_fp8_block(const void* a, int64_t lda, const float* a_scale, int64_t ldas,
                      const void* b, int64_t ldb, const float* b_scale, int64_t ldbs, void* c,
                      int64_t ldc, int out_type, int64_t M, int64_t K, int64_t N, void* stream)
{
    return run_fp8(a, lda, a_scale, ldas, b, ldb, 0, b_scale, ldbs, 0, nullptr, 1, c, ldc,
                   out_type, M, K, N, stream);
}

int ag_gemm_grouped_fp8_block(const void* a, int64_t lda, const float* a_scale, int64_t ldas,
                              const void* b, int64_t ldb, int64_t b_stride, const float* b_scale,
                              int64_t ldbs, int64_t bs_stride, const int32_t* offsets,
                              int n_groups, void* c, int64_t ldc, int out_type, int64_t T,
                              int64_t K, int64_t N, void* stream)
{
    if (!offsets) return AGG_E_INVALID;
    if (!aligned(offsets, 4)) return AGG_E_UNSUPPORTED;
    return run_fp8(a, lda, a_scale, ldas, b, ldb, b_stride, b_scale, ldbs, bs_stride, offsets,
                   n_groups, c, ldc, out_type, T, K, N, stream);
}

int ag_gemm_quant_fp8_block(int type, const void* x, int64_t ldx, void* q, int64_t ldq,
                            float* scale, int64_t lds, int block_rows, int64_t M, int64_t K,
                            void* stream)
{
    int rc = check_sizes(M, K, 1, 1);
    if (rc) return rc;
    if (!is16(type) && type != kTypeF32) return AGG_E_INVALID;
    if (block_rows != 1 && block_rows != kScaleBlock) return AGG_E_INVALID;
    const int64_t kb = (K + kScaleBlock - 1) / kScaleBlock;
    rc = first_error({check_matrix(x, M, K, ldx, elt_of(type)), check_matrix(q, M, K, ldq, 1),
                      check_matrix(scale, M, kb, lds, 4)});
    if (rc) return rc;
    if (M == 0) return AGG_OK;
    const QuantArgs a{static_cast<const char*>(x), static_cast<uint8_t*>(q), scale, M, K,
                      ldx, ldq, lds};
    // 16-byte loads and 8-byte stores of whole pieces
    const bool wide = K % 8 == 0 && ldx * elt_of(type) % 16 == 0 && ldq % 8 == 0 &&
                      aligned(x, 16) && aligned(q, 8);
    return status_of(launch_quant(a, type, block_rows, wide, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
