// launch.hpp -- host side: grids of the grouped kernels and the LDS opt-in.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "experts.hpp"
#include "groups.hpp"

namespace agg {

namespace {

// Workgroups for `tiles` tiles at most, rounded up so that every XCD is
// dealt as many; 0: more threads than one launch can have.
inline uint32_t grid_of(int64_t tiles, int threads)
{
    const int64_t n = (tiles + kXcds - 1) / kXcds * kXcds;
    return n * threads > 0xffffffffll ? 0 : (uint32_t)n;
}

// Row tiles of bi rows that any offsets can need: each group at most one
// more than its rows fill.
inline int64_t row_tiles(const ProductArgs& a, int bi)
{
    const int64_t whole = a.rows / bi;
    const int64_t more = a.groups < a.rows ? a.groups : a.rows;
    return a.offsets ? whole + more : ((int64_t)a.rows + bi - 1) / bi;
}

// More than 64 KiB of LDS is asked for once per kernel and device (`done`:
// one bit a device).
inline hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace

}  // namespace agg
