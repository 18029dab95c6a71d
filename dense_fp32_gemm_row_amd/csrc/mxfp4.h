// Internal declarations of the MXFP4 operators (include/gemm_mxfp4.h).
// Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "mxfp4_choice.h"

namespace gemm_f32_impl {
namespace mx {

// One matrix (of a batch) in the format; strides in bytes.
struct View {
    const uint8_t *codes;
    int64_t ldq, sq;
    const uint8_t *scales;
    int64_t lds, ss;
};
struct Out {
    uint8_t *codes;
    int64_t ldq, sq;
    uint8_t *scales;
    int64_t lds, ss;
};

struct Quantize {
    int64_t batch;
    int rows, cols;
    const float *X;
    int64_t ldx, sx;
    bool along_rows, along_cols;
    Out q, qt;
};
struct Dequantize {
    int64_t batch;
    int rows, cols;
    View q;
    float *Y;
    int64_t ldy, sy;
};
// C = A B^T, or C = A op(W) with A in FP32 (x, ldx, sx in floats).
struct Product {
    int64_t batch;
    int M, N, K;
    View a;
    const float *x;
    int64_t ldx, sx;
    View b;
    bool b_transposed;  // weight product: W is N x K
    float *C;
    int64_t ldc, sc;
    float *W;       // partial sums, or null
    int splits;     // slices of K (1: none)
};

hipError_t launch_quantize(const Quantize &, hipStream_t);
hipError_t launch_dequantize(const Dequantize &, hipStream_t);
hipError_t launch_product(const Product &, hipStream_t);
hipError_t launch_weight(const Product &, hipStream_t);

// Slices of K that launch_product / launch_weight use when they have a
// workspace (1: they need none).
int product_splits(int64_t batch, int64_t M, int64_t N, int64_t K);
int weight_splits(bool b_transposed, int64_t batch, int64_t M, int64_t N, int64_t K);

// C_b = sum over s < splits of slice [b][s] of p.W, in that order.
hipError_t launch_sum_slices(const Product &p, hipStream_t);
}  // namespace mx
}  // namespace gemm_f32_impl
