// Internal declarations of the MXFP4 operators (include/gemm_mxfp4.h).
// Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gemm_f32_impl {
namespace mx {

constexpr int kBlock = 32;        // values that share a scale
constexpr int kBlockBytes = 16;   // their codes

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
// Predicted microseconds of that.
inline double sum_slices_us(double batch, double M, double N, int splits) {
    return splits > 1 ? 4.0 + batch * M * N * 4.0 * (splits + 1) / 3.5e6 : 0.0;
}

// Slices of K of `chunks` chunks each are equally long but for the last: with
// `want` asked for, the number that is not empty.
inline int slices_used(int64_t chunks, int64_t want) {
    const int64_t len = (chunks + want - 1) / want;
    return static_cast<int>((chunks + len - 1) / len);
}

inline int64_t blocks_of(int64_t k) { return (k + kBlock - 1) / kBlock; }

}  // namespace mx
}  // namespace gemm_f32_impl
