// checks.hpp -- host side: what the C entry points check of their arguments
// (before any HIP call), and what they ask of the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "aggemm.h"
#include "experts.hpp"

namespace agg {

namespace {

constexpr int64_t kMaxDim = 1 << 20;           // K, N
constexpr int64_t kMaxLd = 1 << 21;            // elements from row to row: 256 rows stay below 2^31 bytes
constexpr int64_t kMaxRows = INT32_MAX - 256;  // offsets are int32
constexpr int64_t kMaxGroups = 1 << 16;

int elt_of(int type) { return type == kTypeF32 ? 4 : type == kTypeFP8 ? 1 : 2; }
bool is16(int type) { return type == kTypeF16 || type == kTypeBF16; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int status_of(hipError_t e)
{
    if (e == hipSuccess) return AGG_OK;
    // the launchers' own answer where one launch cannot hold the tiles
    if (e == hipErrorInvalidConfiguration) return AGG_E_UNSUPPORTED;
    return AGG_E_HIP;
}

// A row-major matrix argument: present unless it has no rows, rows that do
// not overlap, aligned to its elements, inside the limits.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int elt)
{
    if (rows > 0 && !p) return AGG_E_INVALID;
    if (ld < cols) return AGG_E_INVALID;
    if (ld > kMaxLd || !aligned(p, (size_t)elt)) return AGG_E_UNSUPPORTED;
    return AGG_OK;
}

int check_sizes(int64_t rows, int64_t K, int64_t N, int64_t groups)
{
    if (rows < 0 || K < 1 || N < 1 || groups < 1) return AGG_E_INVALID;
    if (rows > kMaxRows || K > kMaxDim || N > kMaxDim || groups > kMaxGroups)
        return AGG_E_UNSUPPORTED;
    return AGG_OK;
}

int first_error(std::initializer_list<int> all)
{
    for (int rc : all)
        if (rc) return rc;
    return AGG_OK;
}

// Compute units of the current device (asked once), a multiple of the XCDs.
int device_cus(int* out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return AGG_E_HIP;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (!n) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return AGG_E_HIP;
        n = n < 8 ? 8 : n / 8 * 8;
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return AGG_OK;
}

// Whether a matrix is made of whole 16-byte pieces.
bool pieces(const void* p, int64_t ld, int64_t stride, int64_t width, int elt)
{
    return aligned(p, 16) && ld * elt % 16 == 0 && stride * elt % 16 == 0 && width * elt % 16 == 0;
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

}  // namespace

}  // namespace agg
