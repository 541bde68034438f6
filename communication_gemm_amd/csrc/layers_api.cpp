// layers_api.cpp -- the C ABI of what stands around the expert products:
// sorting by expert and back, the norm, microscaled 4-bit values.  Argument
// checks (before any HIP call) and the choice of kernel.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "aggemm.h"
#include "checks.hpp"
#include "layers.hpp"

namespace agg {
namespace {

constexpr int kMaxTop = 1024;

bool is_float(int type) { return is16(type) || type == kTypeF32; }

// Tokens and the rows they have in the order of the experts.
int check_route(int64_t tokens, int top, int64_t rows)
{
    if (tokens < 0 || top < 1 || rows < 0) return AGG_E_INVALID;
    if (top > kMaxTop || tokens > kMaxRows || tokens * top > kMaxRows || rows > kMaxRows)
        return AGG_E_UNSUPPORTED;
    return AGG_OK;
}

int check_place(const int32_t* place, int64_t tokens)
{
    if (tokens > 0 && !place) return AGG_E_INVALID;
    return aligned(place, 4) ? AGG_OK : AGG_E_UNSUPPORTED;
}

// A vector of k values: absent where that is allowed, aligned.
int check_vector(const void* p, int elt, bool wanted)
{
    if (wanted && !p) return AGG_E_INVALID;
    return aligned(p, (size_t)elt) ? AGG_OK : AGG_E_UNSUPPORTED;
}

// A matrix that may be absent.
int check_optional(const void* p, int64_t rows, int64_t cols, int64_t ld, int elt)
{
    return p ? check_matrix(p, rows, cols, ld, elt) : AGG_OK;
}

bool pieces_or_none(const void* p, int64_t ld, int64_t width, int elt)
{
    return !p || pieces(p, ld, 0, width, elt);
}

// Rows of codes: k values, two a byte.
int check_codes(const void* p, int64_t rows, int64_t k, int64_t ld)
{
    return check_matrix(p, rows, k / 2, ld, 1);
}

// The kernel of a 4-bit product, from the sizes the host knows (the groups'
// rows as pick() in experts_api.cpp takes them).  us, weights from HBM:
//   few rows, or a narrow product: 16 rows while a round of workgroups holds
//     all its tiles.  K 7168, N 4096, 5 / 16 rows: 16 rows 6.1 / 6.7, 32 rows
//     6.9 / 7.7, 64 x 64 15; 32 rows, N 2048: 6.8, 8.8; 250 rows, K 4096, N 256:
//     5.5, split 32 x 32 6.5.  Of groups a CU holds several: 3 of 5, K 2048, N
//     2048 (384 tiles) 5.7, 64 x 64 7.1; 8 groups, K 4096 (1024) 12.8, 10.4;
//   then 32 rows in the same way, of more than 32 only where r is short: 32
//     rows, K 7168, N 4096: 8.9, 16 rows 10.7; 64 rows, N 2048, K 2048: 5.2, split
//     32 x 32 5.7; 100 rows, N 1024, K 7168: 8.9, 7.7;
//   up to a round of small tiles, r shared by the groups of a workgroup's waves
//     unless it is short.  32 x 32 / 32 x 64 / 64 x 64 / 64 x 64 not shared: 33
//     rows, K 7168, N 4096: 8.8 / 9.4 / 11.4 / 14.3; 128 rows, K 4096, N 4096:
//     12.9 / 7.7 / 8.9 / 10.0; 256 rows: - / 13.8 / 9.3 / 10.5; 256 rows, K 1024,
//     N 1024: 5.8 / 5.8 / 5.5 / 5.2.  64 x 128: 512 rows, K 4096, N 4096 / 1024
//     rows, K 7168, N 2048: 12.2 / 16.7, 64 x 64 13.0 / 18.4, 128 x 128 14.3 /
//     20.8; 300 rows, K 2048, N 6144: 8.9, 8.5.  8 groups, K 4096, N 4096, mean 5
//     / 25: 64 x 128 16.4 / 17.6, 64 x 64 15.1 / 17.0, 64 x 256 18.4 / 20.3;
//   many groups of few rows.  E 32, K 4096, N 2048, mean 3 / 8 / 25: 64 x 256
//     26.3 / 30.6 / 31.9, 128 x 128 27.5 / 30.4 / 32.6, 64 x 64 30 / 35 / 36; K
//     2048, N 2816, mean 47 / 94: 28.9 / 38.2, 30.7 / 35.3, 35 / 42;
//   and where a round holds those tiles and not the next: 8 groups, K 4096, N
//     2048, mean 200: 17.0, 128 x 128 22.9, large 20.2; 24, K 3584, N 1024, mean 125:
//     16.7, 15.6, 19.4; 32, K 1024, N 1024, mean 81: 8.6, 10.7, 10.4;
//   many, 128 x 128 / large: N 4096, K 4096, 1024 / 2048 / 4096 rows 15.9 / 26.5
//     / 49.2, 19.9 / 24.5 / 37.6; E 8, N 2048, mean 250: 23.7, 20.6; E 32, K
//     2048, N 2816, mean 94: 35.7, 39.8.
int pick_mx(const MxArgs& a, bool whole)
{
    if (!whole) return kAnyLayout;
    const int64_t used = a.groups < a.rows ? a.groups : a.rows;
    const int64_t mean = tiles_of(a.rows, used);
    const int64_t rows = used == 1 ? mean : mean + mean / 4;
    const int64_t strips = used * tiles_of(a.J, 16);
    if (rows <= 16 && (used == 1 || strips <= 2 * a.cus)) return kSkinny16;
    if (tiles_of(rows, 16) * strips <= a.cus) return kSkinny16;
    if (tiles_of(rows, 32) * strips <= a.cus && (rows <= 32 || a.R <= 2048)) return kSkinny32;
    // small tiles: of each group half of one is likely empty
    const auto small = [&](int bi, int bj) {
        const int64_t half = used == 1 ? 0 : used * bi / 2, t = tiles_of(a.rows + half, bi);
        return (t > used ? t : used) * tiles_of(a.J, bj);
    };
    if (a.R > 1024) {
        if (small(32, 32) <= a.cus) return kSplit32x32;
        if (small(32, 64) <= a.cus) return kSplit32x64;
        if (small(64, 64) <= a.cus) return kSplit64x64;
        if (small(64, 128) <= a.cus && mean > 32 && a.R >= 4096) return kSplit64x128;
    }
    if (small(64, 64) <= 2 * a.cus) return kTile64x64;
    if (mean <= 64 && used * tiles_of(a.J, 256) >= 128) return kTile64x256;
    if (small(128, 128) > a.cus && small(64, 256) <= a.cus / 16 * 15) return kTile64x256;
    if (rows > 128 && a.c_pieces && used * tiles_of(rows, 128) * tiles_of(a.J, 256) >= 160) return kTileLarge;
    return kTile128x128;
}

int run_mx(const void* a, int64_t lda, const uint8_t* as, int64_t ldas, const void* b, int64_t ldb,
           int64_t b_stride, const uint8_t* bs, int64_t ldbs, int64_t bs_stride, const int32_t* offsets,
           int64_t groups, void* c, int64_t ldc, int out_type, int64_t M, int64_t K, int64_t N, void* stream)
{
    int rc = check_sizes(M, K, N, groups);
    if (rc) return rc;
    if (!is_float(out_type) || K % 2) return AGG_E_INVALID;
    const int64_t kb = (K + kMxBlock - 1) / kMxBlock;
    rc = first_error({check_codes(a, M, K, lda), check_matrix(as, M, kb, ldas, 1), check_codes(b, N, K, ldb),
                      check_matrix(bs, N, kb, ldbs, 1), check_matrix(c, M, N, ldc, elt_of(out_type))});
    if (rc) return rc;
    if (b_stride < 0 || bs_stride < 0) return AGG_E_INVALID;
    if (M == 0) return AGG_OK;
    MxArgs p{};
    p.p = static_cast<const char*>(a);
    p.q = static_cast<const char*>(b);
    p.c = static_cast<char*>(c);
    p.pe = as;
    p.qe = bs;
    p.offsets = offsets;
    p.rows = (int)M;
    p.groups = (int)groups;
    p.ldp = lda;
    p.ldq = ldb;
    p.ldc = ldc;
    p.q_stride = b_stride;
    // a single row's stride is not looked at: one that keeps rows on dwords
    p.ldps = M == 1 ? (ldas + 3) / 4 * 4 : ldas;
    p.ldqs = N == 1 ? (ldbs + 3) / 4 * 4 : ldbs;
    p.qs_stride = bs_stride;
    p.J = (int)N;
    p.R = (int)K;
    p.out_type = out_type;
    rc = device_cus(&p.cus);
    if (rc) return rc;
    const bool whole = pieces(a, lda, 0, K / 2, 1) && pieces(b, ldb, b_stride, K / 2, 1);
    p.c_pieces = pieces(c, ldc, 0, N, elt_of(out_type));
    const bool dwords = aligned(as, 4) && aligned(bs, 4) && p.ldps % 4 == 0 && p.ldqs % 4 == 0 && bs_stride % 4 == 0;
    return status_of(launch_mx(p, pick_mx(p, whole), !dwords, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace agg

using namespace agg;

extern "C" {

size_t ag_gemm_expert_sort_workspace_bytes(int64_t T, int top, int n_experts)
{
    if (check_route(T, top, 0) || n_experts < 1 || n_experts > kMaxExperts) return 0;
    const int64_t n = T * top;
    return n > kSortRecount ? (size_t)sort_blocks(n) * n_experts * 4 : 0;
}

int ag_gemm_expert_sort(const void* ids, int id_bytes, int64_t ldi, int64_t T, int top, int n_experts,
                        int32_t* offsets, int32_t* place, void* workspace, size_t workspace_bytes,
                        void* stream)
{
    int rc = check_route(T, top, 0);
    if (rc) return rc;
    if ((id_bytes != 4 && id_bytes != 8) || n_experts < 1 || !offsets) return AGG_E_INVALID;
    if (n_experts > kMaxExperts) return AGG_E_UNSUPPORTED;
    rc = first_error({check_matrix(ids, T, top, ldi, id_bytes), check_place(place, T),
                      check_vector(offsets, 4, true)});
    if (rc) return rc;
    const size_t need = ag_gemm_expert_sort_workspace_bytes(T, top, n_experts);
    if (need && (!workspace || workspace_bytes < need)) return AGG_E_INVALID;
    if (need && !aligned(workspace, 4)) return AGG_E_UNSUPPORTED;
    const SortArgs a{ids, ldi, offsets, place, static_cast<int32_t*>(workspace), (int)(T * top), top, n_experts,
                     sort_chunk(T * top)};
    return status_of(launch_sort(a, id_bytes == 8, static_cast<hipStream_t>(stream)));
}

int ag_gemm_expert_dispatch(int type, const void* x, int64_t ldx, const int32_t* place, int top, void* xs,
                            int64_t ldxs, int64_t rows, int64_t T, int64_t K, void* stream)
{
    int rc = first_error({check_route(T, top, rows), check_sizes(T, K, 1, 1)});
    if (rc) return rc;
    if (!is_float(type) && type != kTypeFP8) return AGG_E_INVALID;
    const int elt = elt_of(type);
    rc = first_error({check_matrix(x, T, K, ldx, elt), check_place(place, T),
                      check_matrix(xs, rows, K, ldxs, elt)});
    if (rc) return rc;
    if (T == 0 || rows == 0) return AGG_OK;
    const DispatchArgs a{static_cast<const char*>(x), static_cast<char*>(xs), place, ldx * elt, ldxs * elt,
                         K * elt, T, top, (int)rows};
    const bool whole = pieces(x, ldx, 0, K, elt) && pieces(xs, ldxs, 0, K, elt);
    return status_of(launch_dispatch(a, whole ? 16 : elt, static_cast<hipStream_t>(stream)));
}

int ag_gemm_expert_combine(int type, const void* h, int64_t ldh, int64_t rows, const int32_t* place, int top,
                           const float* w, int64_t ldw, void* y, int64_t ldy, int out_type, int64_t T,
                           int64_t K, void* stream)
{
    int rc = first_error({check_route(T, top, rows), check_sizes(T, K, 1, 1)});
    if (rc) return rc;
    if (!is_float(type) || (out_type != type && out_type != kTypeF32)) return AGG_E_INVALID;
    rc = first_error({check_matrix(h, rows, K, ldh, elt_of(type)), check_place(place, T),
                      check_optional(w, T, top, ldw, 4), check_matrix(y, T, K, ldy, elt_of(out_type))});
    if (rc) return rc;
    if (T == 0) return AGG_OK;
    CombineArgs a{};
    a.h = static_cast<const char*>(h);
    a.place = place;
    a.w = w;
    a.y = static_cast<char*>(y);
    a.ldh = ldh;
    a.ldw = ldw;
    a.ldy = ldy;
    a.tokens = T;
    a.k = K;
    a.top = top;
    a.rows = (int)rows;
    const bool wide = pieces(h, ldh, 0, 8, elt_of(type)) && pieces(y, ldy, 0, 8, elt_of(out_type)) && K % 8 == 0;
    return status_of(launch_combine(a, type, out_type, wide, static_cast<hipStream_t>(stream)));
}

int ag_gemm_expert_combine_grad(int type, const void* dy, int64_t lddy, const void* h, int64_t ldh, int64_t rows,
                                const int32_t* place, int top, const float* w, int64_t ldw, void* dh,
                                int64_t lddh, float* dw, int64_t lddw, int64_t T, int64_t K, void* stream)
{
    int rc = first_error({check_route(T, top, rows), check_sizes(T, K, 1, 1)});
    if (rc) return rc;
    if (!is_float(type) || (!dh && !dw && T > 0 && rows > 0)) return AGG_E_INVALID;
    const int elt = elt_of(type);
    rc = first_error({check_matrix(dy, T, K, lddy, elt), check_place(place, T), check_matrix(w, T, top, ldw, 4),
                      dw ? check_matrix(h, rows, K, ldh, elt) : (int)AGG_OK,
                      check_optional(dh, rows, K, lddh, elt), check_optional(dw, T, top, lddw, 4)});
    if (rc) return rc;
    if (T == 0) return AGG_OK;
    CombineArgs a{};
    a.h = static_cast<const char*>(h);
    a.place = place;
    a.w = w;
    a.y = static_cast<char*>(const_cast<void*>(dy));
    a.dh = static_cast<char*>(dh);
    a.dw = dw;
    a.ldh = ldh;
    a.ldw = ldw;
    a.ldy = lddy;
    a.lddh = lddh;
    a.lddw = lddw;
    a.tokens = T;
    a.k = K;
    a.top = top;
    a.rows = (int)rows;
    const bool wide = K % 8 == 0 && pieces(dy, lddy, 0, 8, elt) && (!dw || pieces(h, ldh, 0, 8, elt)) &&
                      pieces_or_none(dh, lddh, 8, elt);
    return status_of(launch_combine_grad(a, type, wide, static_cast<hipStream_t>(stream)));
}

int ag_gemm_rmsnorm(int type, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                    void* h, int64_t ldh, void* y, int64_t ldy, void* q, int64_t ldq, float* scale, int64_t lds,
                    float* rstd, float eps, int64_t T, int64_t K, void* stream)
{
    int rc = check_sizes(T, K, 1, 1);
    if (rc) return rc;
    if (!is_float(type) || !(eps >= 0.f) || isinf(eps)) return AGG_E_INVALID;
    if (T > 0 && ((!y && !q) || (!q) != (!scale))) return AGG_E_INVALID;
    const int elt = elt_of(type);
    const int64_t kb = (K + kScaleBlock - 1) / kScaleBlock;
    rc = first_error({check_matrix(x, T, K, ldx, elt), check_optional(residual, T, K, ldr, elt),
                      check_vector(weight, elt, false), check_optional(h, T, K, ldh, elt),
                      check_optional(y, T, K, ldy, elt), check_optional(q, T, K, ldq, 1),
                      check_optional(scale, T, kb, lds, 4), check_vector(rstd, 4, false)});
    if (rc) return rc;
    // h in the place of x or of the residual: the same rows
    if (h && ((h == x && ldh != ldx && T > 1) || (h == residual && ldh != ldr && T > 1))) return AGG_E_INVALID;
    if (T == 0) return AGG_OK;
    const NormArgs a{static_cast<const char*>(x), static_cast<const char*>(residual),
                     static_cast<const char*>(weight), static_cast<char*>(h), static_cast<char*>(y),
                     static_cast<uint8_t*>(q), scale, rstd, ldx, ldr, ldh, ldy, ldq, lds, T, K, eps};
    const bool wide = K % 8 == 0 && pieces(x, ldx, 0, 8, elt) && pieces_or_none(residual, ldr, 8, elt) &&
                      aligned(weight, 16) && pieces_or_none(h, ldh, 8, elt) && pieces_or_none(y, ldy, 8, elt) &&
                      (!q || (aligned(q, 8) && ldq % 8 == 0));
    return status_of(launch_norm(a, type, wide, static_cast<hipStream_t>(stream)));
}

size_t ag_gemm_rmsnorm_grad_workspace_bytes(int64_t T, int64_t K)
{
    if (check_sizes(T, K, 1, 1)) return 0;
    return (size_t)norm_grad_parts(T) * K * 4;
}

int ag_gemm_rmsnorm_grad(int type, const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                         const float* rstd, const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dw,
                         int dw_type, void* workspace, size_t workspace_bytes, int64_t T, int64_t K,
                         void* stream)
{
    int rc = check_sizes(T, K, 1, 1);
    if (rc) return rc;
    if (!is_float(type) || (dw && dw_type != type && dw_type != kTypeF32)) return AGG_E_INVALID;
    const int elt = elt_of(type);
    rc = first_error({check_matrix(dy, T, K, lddy, elt), check_matrix(h, T, K, ldh, elt),
                      check_vector(weight, elt, false), check_vector(rstd, 4, T > 0),
                      check_optional(dh, T, K, lddh, elt), check_matrix(dx, T, K, lddx, elt),
                      check_vector(dw, dw ? elt_of(dw_type) : 1, false)});
    if (rc) return rc;
    const size_t need = dw ? ag_gemm_rmsnorm_grad_workspace_bytes(T, K) : 0;
    if (need && (!workspace || workspace_bytes < need)) return AGG_E_INVALID;
    if (need && !aligned(workspace, 16)) return AGG_E_UNSUPPORTED;
    if (T == 0 && !dw) return AGG_OK;
    const NormGradArgs a{static_cast<const char*>(dy), static_cast<const char*>(h),
                         static_cast<const char*>(weight), rstd, static_cast<const char*>(dh),
                         static_cast<char*>(dx), static_cast<char*>(dw), static_cast<float*>(workspace),
                         lddy, ldh, lddh, lddx, T, K, norm_grad_parts(T), dw_type};
    const bool wide = K % 8 == 0 && pieces(dy, lddy, 0, 8, elt) && pieces(h, ldh, 0, 8, elt) &&
                      aligned(weight, 16) && pieces_or_none(dh, lddh, 8, elt) && pieces(dx, lddx, 0, 8, elt);
    return status_of(launch_norm_grad(a, type, wide, static_cast<hipStream_t>(stream)));
}

int ag_gemm_quant_mxfp4(int type, const void* x, int64_t ldx, void* q, int64_t ldq, uint8_t* scale, int64_t lds,
                        int64_t M, int64_t K, void* stream)
{
    int rc = check_sizes(M, K, 1, 1);
    if (rc) return rc;
    if (!is_float(type) || K % 2) return AGG_E_INVALID;
    const int elt = elt_of(type);
    const int64_t kb = (K + kMxBlock - 1) / kMxBlock;
    rc = first_error({check_matrix(x, M, K, ldx, elt), check_codes(q, M, K, ldq), check_matrix(scale, M, kb, lds, 1)});
    if (rc) return rc;
    if (M == 0) return AGG_OK;
    const MxQuantArgs a{static_cast<const char*>(x), static_cast<uint8_t*>(q), scale, M, K, ldx, ldq, lds};
    const bool wide = K % 8 == 0 && pieces(x, ldx, 0, 8, elt) && aligned(q, 4) && ldq % 4 == 0;
    return status_of(launch_mx_quant(a, type, wide, static_cast<hipStream_t>(stream)));
}

int ag_gemm_dequant_mxfp4(const void* q, int64_t ldq, const uint8_t* scale, int64_t lds, void* y, int64_t ldy,
                          int type, int64_t M, int64_t K, void* stream)
{
    int rc = check_sizes(M, K, 1, 1);
    if (rc) return rc;
    if (!is_float(type) || K % 2) return AGG_E_INVALID;
    const int elt = elt_of(type);
    const int64_t kb = (K + kMxBlock - 1) / kMxBlock;
    rc = first_error({check_codes(q, M, K, ldq), check_matrix(scale, M, kb, lds, 1), check_matrix(y, M, K, ldy, elt)});
    if (rc) return rc;
    if (M == 0) return AGG_OK;
    const MxQuantArgs a{static_cast<const char*>(y), static_cast<uint8_t*>(const_cast<void*>(q)),
                        const_cast<uint8_t*>(scale), M, K, ldy, ldq, lds};
    const bool wide = K % 8 == 0 && pieces(y, ldy, 0, 8, elt) && aligned(q, 4) && ldq % 4 == 0;
    return status_of(launch_mx_dequant(a, type, wide, static_cast<hipStream_t>(stream)));
}

int ag_gemm_mxfp4(const void* a, int64_t lda, const uint8_t* a_scale, int64_t ldas, const void* b, int64_t ldb,
                  const uint8_t* b_scale, int64_t ldbs, void* c, int64_t ldc, int out_type, int64_t M,
                  int64_t K, int64_t N, void* stream)
{
    return run_mx(a, lda, a_scale, ldas, b, ldb, 0, b_scale, ldbs, 0, nullptr, 1, c, ldc, out_type, M, K, N,
                  stream);
}

int ag_gemm_grouped_mxfp4(const void* a, int64_t lda, const uint8_t* a_scale, int64_t ldas, const void* b,
                          int64_t ldb, int64_t b_stride, const uint8_t* b_scale, int64_t ldbs,
                          int64_t bs_stride, const int32_t* offsets, int n_groups, void* c, int64_t ldc,
                          int out_type, int64_t T, int64_t K, int64_t N, void* stream)
{
    if (!offsets) return AGG_E_INVALID;
    if (!aligned(offsets, 4)) return AGG_E_UNSUPPORTED;
    return run_mx(a, lda, a_scale, ldas, b, ldb, b_stride, b_scale, ldbs, bs_stride, offsets, n_groups, c, ldc,
                  out_type, T, K, N, stream);
}

}  // extern "C"
