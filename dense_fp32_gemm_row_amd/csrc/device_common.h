// Device helpers shared by the MXFP4 and the fused operators.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gemm_f32_impl {

typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));  // 16 bytes at any word
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Waits until at most N of this wavefront's most recent vector-memory
// instructions and no LDS access are outstanding.  The empty asm statements
// keep memory accesses on their side.
template <int N>
__device__ __forceinline__ void wait_older() {
    static_assert(N >= 0 && N < 64, "vmcnt has 6 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier_only() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace gemm_f32_impl
