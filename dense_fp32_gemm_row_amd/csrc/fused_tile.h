// The tile kernel of the fused products: C = epilogue(op(A) op(B)), or the row
// statistics of the cross entropy, for a tile of C that a workgroup holds in
// registers.  Each operand form is compiled in a source file of its own.
#pragma once

#include <type_traits>

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {

// LDS holds rows (of op(A), columns of op(B)) in groups of 64 in an order of
// its own: place 32 f + 16 h + i of a group is row 4 i + 2 h + f.  A lane
// that takes places j and 32 + j of a group so holds two neighbouring columns
// of C, and its half wavefront 64 of them, which are stored as a piece; and a lane that
// stages 4 neighbouring rows writes to 4 places 16 apart, next to its
// neighbours'.
__device__ __forceinline__ int row_at(int place) {
    return (place & ~63) + 4 * (place & 15) + ((place >> 3) & 2) + ((place >> 5) & 1);
}
__device__ __forceinline__ int place_of_row(int row) {
    return (row & ~63) + ((row >> 2) & 15) + ((row & 2) << 3) + ((row & 1) << 5);
}

template <int WM, int WN, int FM>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int BM = 32 * FM * WM, BN = 64 * WN;
};

// Elements of one k range of an operand's tile, rows and k past the end zero.
// KC: k is contiguous (A as stored, B transposed).
template <bool KC>
__device__ __forceinline__ float element(const float *p, int64_t ld, int row, int rows, int k, int k1) {
    if (row >= rows || k >= k1) return 0.0f;
    return KC ? p[row * ld + k] : p[k * ld + row];
}

template <int WM, int WN, int FM, bool TA, bool TB>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(Product p, int tiles_m, int tiles_n,
                                                             int64_t tiles, int len) {
    using T = Tile<WM, WN, FM>;
    constexpr int BM = T::BM, BN = T::BN, kThreads = T::kThreads;
    __shared__ __align__(16) float xs[kStage][BM];
    __shared__ __align__(16) float ys[kStage][BN];

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    const int64_t per = static_cast<int64_t>(tiles_m) * tiles_n;
    for (int64_t id = xcd_remap(blockIdx.x, gridDim.x); id < tiles; id += gridDim.x) {
        const int64_t slice = id / per, b = slice / p.splits;
        int tm, tn;
        grouped_tile(static_cast<int>(id - slice * per), tiles_m, tiles_n, 8, tm, tn);
        const int m0 = tm * BM, n0 = tn * BN;
        const int k0 = static_cast<int>(slice - b * p.splits) * len;
        const int k1 = static_cast<int>(min(static_cast<int64_t>(k0) + len, static_cast<int64_t>(p.K)));
        const float *A = p.a.p + b * p.a.stride + (TA ? m0 : m0 * p.a.ld);
        const float *B = p.b.p + b * p.b.stride + (TB ? n0 * p.b.ld : n0);
        const int rows = p.M - m0, cols = p.N - n0;

        f32x16 acc[FM][2];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) acc[i][f] = f32x16{};
        };

        // FP32 multiplies: any shape, any value, one stage at a time.
        auto general = [&](int first, int last, const int64_t *skip) {
            for (int k = first; k < last; k += kStage) {
                __syncthreads();
                for (int o = tid; o < BM * kStage; o += kThreads) {
                    const int r = TA ? o % BM : o / kStage, q = TA ? o / BM : o % kStage;
                    float v = element<!TA>(A, p.a.ld, r, rows, k + q, last);
                    if (skip != nullptr && k + q < last && skip[k + q] == p.ignore_k) v = 0.0f;
                    xs[q][place_of_row(r)] = v;
                }
                for (int o = tid; o < BN * kStage; o += kThreads) {
                    const int r = TB ? o / kStage : o % BN, q = TB ? o % kStage : o / BN;
                    float v = element<TB>(B, p.b.ld, r, cols, k + q, last);
                    if (skip != nullptr && k + q < last && skip[k + q] == p.ignore_k) v = 0.0f;
                    ys[q][place_of_row(r)] = v;
                }
                __syncthreads();
#pragma unroll
                for (int q = 0; q < kStage; q += 2) {
                    float y[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f) y[f] = ys[q + half][64 * wn + 32 * f + col];
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const float x = xs[q + half][32 * (FM * wm + i) + col];
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y[f], acc[i][f], 0, 0, 0);
                    }
                }
            }
            __syncthreads();
        };

        clear();
        general(k0, k1, p.target_k);

        // ---- results: a lane has two neighbouring columns of FM * 16 rows ----
        const int n = n0 + 64 * wn + 4 * (col & 15) + 2 * (col >> 4);
        // row r of block i, from the wavefront's first
        auto row_of = [&](int i, int r) {
            return row_at(32 * (FM * wm + i) + (r & 3) + 8 * (r >> 2) + 4 * half);
        };
        auto put = [&](float *dst, int64_t at, float v0, float v1) {
            if (n + 1 < p.N)
                *reinterpret_cast<float2u *>(dst + at) = float2u{v0, v1};
            else
                dst[at] = v0;
        };
        auto get = [&](const float *src, int64_t at) {
            return n + 1 < p.N ? *reinterpret_cast<const float2u *>(src + at) : float2u{src[at], 0.0f};
        };
        if (p.mode != kStore) {
            const int group = tn * WN + wn;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int m = m0 + row_of(i, r);
                    const float v0 = n < p.N ? acc[i][0][r] : -__builtin_inff();
                    const float v1 = n + 1 < p.N ? acc[i][1][r] : -__builtin_inff();
                    float top = fmaxf(v0, v1);
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
                    const float base = top == -__builtin_inff() ? 0.0f : top;
                    float s = expf(v0 - base) + expf(v1 - base);
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) s += __shfl_xor(s, d);
                    if (m < p.M) {
                        if (n0 + 64 * wn < p.N && col == 0)
                            p.stats[static_cast<int64_t>(m) * p.groups + group] = stat2{top, s};
                        const int64_t t = p.target[m] - n;
                        if (t == 0 && n < p.N) p.at_target[m] = v0;
                        if (t == 1 && n + 1 < p.N) p.at_target[m] = v1;
                        if (p.mode == kStoreStats && n < p.N) put(p.c.p, m * p.c.ld + n, v0, v1);
                    }
                }
            continue;
        }
        if (n >= p.N) continue;
        if (p.splits > 1) {
            float *W = p.slices + slice * p.M * p.N;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t m = m0 + row_of(i, r);
                    if (m < p.M) put(W, m * p.N + n, acc[i][0][r], acc[i][1][r]);
                }
            continue;
        }
        float2u bias{0.0f, 0.0f};
        if (p.e.bias.p != nullptr) bias = get(p.e.bias.p + b * p.e.bias.stride, n);
        float *C = p.c.p + b * p.c.stride, *Z = p.e.pre.p + b * p.e.pre.stride;
        const float *R = p.e.residual.p + b * p.e.residual.stride;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t m = m0 + row_of(i, r);
                if (m >= p.M) continue;
                const float z0 = acc[i][0][r] + bias[0], z1 = acc[i][1][r] + bias[1];
                if (p.e.pre.p != nullptr) put(Z, m * p.e.pre.ld + n, z0, z1);
                float v0 = activate(p.e.activation, z0), v1 = activate(p.e.activation, z1);
                if (p.e.residual.p != nullptr) {
                    const float2u q = get(R, m * p.e.residual.ld + n);
                    v0 += q[0], v1 += q[1];
                }
                put(C, m * p.c.ld + n, v0, v1);
            }
    }
}

template <int WM, int WN, int FM, bool TA, bool TB>
hipError_t launch_one(const Product &p, hipStream_t stream) {
    using T = Tile<WM, WN, FM>;
    const int tm = static_cast<int>(div_up(p.M, T::BM)), tn = static_cast<int>(div_up(p.N, T::BN));
    const int64_t tiles = static_cast<int64_t>(tm) * tn * p.batch * p.splits;
    // whole stages a slice
    const int len = static_cast<int>(div_up(div_up(p.K, kStage), p.splits)) * kStage;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 21));
    tile_kernel<WM, WN, FM, TA, TB><<<grid, T::kThreads, 0, stream>>>(p, tm, tn, tiles, len);
    return hipGetLastError();
}

template <bool TA, bool TB>
hipError_t launch_tile(const Product &p, int tile, hipStream_t stream) {
    (void)tile;
    return launch_one<2, 2, 1, TA, TB>(p, stream);
}

}  // namespace fused
}  // namespace gemm_f32_impl
