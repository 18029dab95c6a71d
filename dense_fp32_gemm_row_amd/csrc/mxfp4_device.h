// Device helpers of the MXFP4 kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gemm_f32_impl {
namespace mx {

typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));  // 16 bytes at any word
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The conversion instructions take a scale as a float and use its exponent
// byte alone: 0 is 2^-127 and 255 NaN, as in the format.
__device__ __forceinline__ float scale_of(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

}  // namespace mx
}  // namespace gemm_f32_impl
