// Internal declarations of the fused operators (include/gemm_f32_fused.h).
// Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fused_choice.h"

namespace gemm_f32_impl {
namespace fused {

typedef float stat2 __attribute__((ext_vector_type(2), aligned(4)));  // (maximum, sum of exponentials)

// One matrix (of a batch); strides in floats.
struct Operand {
    const float *p;
    int64_t ld, stride;
};
struct Result {
    float *p;
    int64_t ld, stride;
};

struct Epilogue {
    int activation;
    Operand bias;      // ld unused
    Operand residual;  // p null: none
    Result pre;        // p null: none
};

// Of one row of op(A) (column of op(B)), or a block of its k: the largest exponent field,
// how many values are not zero, and the sum of their exponent fields.
struct RowStat {
    int top, count, sum, unused;
};

// What the tile kernel does with a tile's sums.
enum Mode : int {  // of a product
    kStore = 0,       // the epilogue (or raw slices), stored
    kStoreSome = 1,   // the same, but rows that take no part are zeros whatever B holds
    kStats = 2,       // a maximum and a sum of exponentials per row and group of columns
    kStoreStats = 3,  // both; the sums are stored as they are
};

// C = epilogue(op(A) op(B)); ta: A is stored K x M, tb: B is stored N x K.
struct Product {
    int64_t batch;
    int M, N, K;
    bool ta, tb;
    Operand a, b;
    Epilogue e;
    Result c;
    bool narrow;    // rows of a tile span less than 2^32 bytes
    float *space;   // product_space() bytes, or null
    // set by launch_product:
    float *slices;  // partial sums [batch][split][M][N], or null
    int splits;     // slices of K (1: none)
    const RowStat *row_a, *row_b;  // [block of k][batch * rows], or null: no fp16 parts
    int blocks_a, blocks_b;
    // kStats, kStoreStats (no batch, no slices): stats[row * groups + column / group_columns(M)];
    // at_target[row] gets the sum in column target[row], where there is one.
    Mode mode;
    stat2 *stats;
    int groups;
    float *at_target;
    const int64_t *target;  // but for kStore: rows m with target[m] == ignore take no part
    // Where not null, k with target_k[k] == ignore, whose factors of A are zero, take
    // no part even where B holds infinities or NaN (A stored K x M, B stored K x N).
    const int64_t *target_k;
    int64_t ignore;
    Use use;
};

hipError_t launch_product(const Product &, hipStream_t);
// Two independent products; they share their workspace, of `bytes`.
hipError_t launch_two(const Product &, const Product &, int64_t bytes, hipStream_t);
// Bytes of workspace that a product is quickest with; it runs with none, too.
int64_t product_space(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, Use use);
// The same of launch_two's.
struct Sizes {
    bool ta, tb;
    int64_t batch, M, N, K;
    Use use;
};
int64_t two_space(const Sizes &, const Sizes &);

// The tile kernels, by operand form (fused_nn.hip ...); `tile` as in
// fused_choice.h.
hipError_t launch_tile_nn(const Product &, int tile, hipStream_t);
hipError_t launch_tile_nt(const Product &, int tile, hipStream_t);
hipError_t launch_tile_tn(const Product &, int tile, hipStream_t);
hipError_t launch_tile_tt(const Product &, int tile, hipStream_t);

// Both in one launch, in tiles of kTiles[1] or [2], p N x N or N x T and q T x N: whether they were.
bool launch_tile_pair(const Product &p, const Product &q, int tile, hipStream_t, hipError_t *err);

// `shape` as in fused_choice.h.
hipError_t launch_rows(const Product &, int shape, hipStream_t);

// Both in one launch, where both are small: whether they were (their splits are
// set; *err is the launch's).
bool launch_rows_pair(const Product &p, int shape_p, const Product &q, int shape_q, hipStream_t, hipError_t *err);

hipError_t launch_row_stats(const Product &, hipStream_t);

// C = epilogue(sum over the slices, in their order).
hipError_t launch_sum_slices(const Product &, hipStream_t);
hipError_t launch_sum_slices(const Product &, const Product &, hipStream_t);  // (the second's mode kStore)

// dZ = dC act'(Z), and the sums of its columns over blocks of rows; either may
// be absent (dz.p null; partial null).
constexpr int kSlopeBlocks = 256;  // at most
struct Slope {
    int64_t batch;
    int M, N;
    int activation;
    Operand dc, pre;
    Result dz;
    float *partial;  // [batch][blocks][N]
    int blocks, rows;  // rows a block; of one block dbias is the sum (partial unused)
    Result dbias;    // ld unused
};
hipError_t launch_slope(const Slope &, hipStream_t);

// The rest of the cross entropy: T rows, row t of `stats` in `groups` pieces.
struct Loss {
    int T, V;
    const stat2 *stats;
    int groups;
    const float *at_target;
    const int64_t *target;
    int64_t ignore;
    float *loss, *lse;          // loss may be null
    const float *grad_loss;     // null: ones
    float *logits;              // launch_probabilities: T x V, in place
    int64_t ld;
};
hipError_t launch_loss(const Loss &, hipStream_t);
// logits = grad_loss (exp(logits - lse) - (v == target)), zero for ignored rows
hipError_t launch_probabilities(const Loss &, hipStream_t);
// Both at once, for small T x V.
hipError_t launch_loss_and_probabilities(const Loss &, hipStream_t);

}  // namespace fused
}  // namespace gemm_f32_impl
