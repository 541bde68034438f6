// device.hpp -- what the expert-product kernels use of the matrix hardware:
// vector types of the matrix instructions, address-space pointers, buffer
// descriptors, waits and the bare workgroup barrier.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace agg {

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef short short4_ __attribute__((ext_vector_type(4)));
#define LDS_PTR __attribute__((address_space(3)))

// Buffer descriptor word 3 for untyped 32-bit accesses, and an offset no
// buffer of this code reaches (range checks return zero for it).
constexpr int kRsrcWord3 = 0x00020000;
constexpr uint32_t kOutOfRange = 0x80000000u;

// s_waitcnt with vmcnt(n), lgkmcnt(0), expcnt untouched (gfx9 encoding).
template <int n>
__device__ __forceinline__ void wait_vm_lgkm0()
{
    static_assert(n >= 0 && n < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
}

// A value that every lane holds alike, marked as such for the compiler.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint64_t u = (uint64_t)v;
    return (int64_t)((uint64_t)uniform((uint32_t)u) | ((uint64_t)uniform((uint32_t)(u >> 32)) << 32));
}

// A buffer descriptor over `bytes` bytes from p (taken as 0 below 0 and as
// 2^31 - 1 above it) in scalar registers: left in vector registers it would
// make the compiler wrap every access in a loop over the lanes' values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scalar_rsrc(const void* p, int64_t bytes)
{
    const int64_t base = uniform((int64_t)reinterpret_cast<uintptr_t>(p));
    const int64_t n = bytes < 0 ? 0 : bytes < 0x7fffffff ? bytes : 0x7fffffff;
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uintptr_t)base), 0,
                                             uniform((int)n), kRsrcWord3);
}

// Workgroup barrier without the release/acquire fences of __syncthreads:
// those would wait for every load still in flight, including the slices
// being prefetched.  Callers wait for exactly what the barrier publishes
// (their own finished loads and LDS reads) before it.  The empty asm
// statements keep the compiler from moving memory accesses across it.
__device__ __forceinline__ void bare_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace

}  // namespace agg
