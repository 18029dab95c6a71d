// The fused products with few rows of op(A): reading B is the work.

#include <type_traits>

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {
namespace {

// A workgroup of 8 wavefronts holds 16 MG rows and 16 NG columns; its
// wavefronts take steps of 64 (32) k in turn, straight from global memory, a step
// ahead, and their sums are added in LDS in a fixed order.  In
// v_mfma_f32_16x16x4_f32 lane l holds one k, l / 16, of row (column) l % 16; here
// lane group g = l / 16 holds k 16 u + 4 g + j of a step in instruction (u, j),
// so its part of A, and of B where that is stored N x K (TB), is 16 bytes of a
// row.  B stored K x N is read NG neighbouring columns at a time.
constexpr int kRowsWaves = 8;
constexpr int quads_of(int mg, int ng) { return (mg + ng) * 4 <= 20 ? 4 : 2; }  // for two steps' registers
template <int MG, int NG, bool TB>
__global__ __launch_bounds__(64 * kRowsWaves) void rows_kernel(Product p, int tiles_n, int64_t tiles, int len) {
    constexpr int kQuads = quads_of(MG, NG), kStep = 16 * kQuads;
    typedef float cols_t __attribute__((ext_vector_type(NG < 2 ? 2 : NG), aligned(4)));
    __shared__ __align__(16) float sums[kRowsWaves][MG * NG][4][64];
    const int lane = threadIdx.x & 63, at = lane & 15, group = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t slice = t / tiles_n, b = slice / p.splits;
        const int n0 = static_cast<int>(t - slice * tiles_n) * 16 * NG;
        const int k0 = static_cast<int>(slice - b * p.splits) * len;
        const int k1 = max(k0, static_cast<int>(min(static_cast<int64_t>(k0) + len, static_cast<int64_t>(p.K))));
        const float *A = p.a.p + b * p.a.stride, *B = p.b.p + b * p.b.stride;
        // rows and columns past the end repeat the last ones' and are not stored
        const float *pa[MG], *pb[TB ? NG : 1];
#pragma unroll
        for (int m = 0; m < MG; ++m) {
            const int64_t r = min(16 * m + at, p.M - 1);
            pa[m] = A + (p.ta ? r : r * p.a.ld);
        }
        // as stored: a lane whose columns pass the end takes the last NG
        const int first = min(n0 + NG * at, p.N - NG);
        if constexpr (TB) {
#pragma unroll
            for (int c = 0; c < NG; ++c) pb[c] = B + static_cast<int64_t>(min(n0 + 16 * c + at, p.N - 1)) * p.b.ld;
        } else {
            pb[0] = B + first;
        }
        struct Step {
            f32x4 a[MG][kQuads];
            f32x4 b[NG][kQuads];
        };
        auto load = [&](int k) {
            Step s;
            const bool whole = k + kStep <= k1;
#pragma unroll
            for (int u = 0; u < kQuads; ++u) {
                const int q = k + 16 * u + 4 * group;
                if constexpr (TB) {
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        if (whole) {
                            s.b[c][u] = *reinterpret_cast<const float4u *>(pb[c] + q);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) s.b[c][u][j] = q + j < k1 ? pb[c][q + j] : 0.0f;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float *from = pb[0] + static_cast<int64_t>(whole ? q + j : min(q + j, k1 - 1)) * p.b.ld;
                        const bool in = whole || q + j < k1;
                        if constexpr (NG == 1) {
                            s.b[0][u][j] = in ? *from : 0.0f;
                        } else {
                            const cols_t v = *reinterpret_cast<const cols_t *>(from);
#pragma unroll
                            for (int c = 0; c < NG; ++c) s.b[c][u][j] = in ? v[c] : 0.0f;
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < MG; ++m) {
                    if (!p.ta && whole) {
                        s.a[m][u] = *reinterpret_cast<const float4u *>(pa[m] + q);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s.a[m][u][j] = whole || q + j < k1 ? pa[m][p.ta ? (q + j) * p.a.ld : q + j] : 0.0f;
                    }
                }
            }
            return s;
        };
        f32x4 acc[MG][NG];
#pragma unroll
        for (int m = 0; m < MG; ++m)
#pragma unroll
            for (int c = 0; c < NG; ++c) acc[m][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        int k = k0 + wave * kStep;
        if (k < k1) {
            Step now = load(k);
            for (;;) {
                const int ahead = k + kRowsWaves * kStep;
                const bool more = ahead < k1;
                Step next;
                if (more) next = load(ahead);
#pragma unroll
                for (int u = 0; u < kQuads; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int m = 0; m < MG; ++m)
#pragma unroll
                            for (int c = 0; c < NG; ++c)
                                acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(now.a[m][u][j], now.b[c][u][j],
                                                                                 acc[m][c], 0, 0, 0);
                if (!more) break;
                now = next;
                k = ahead;
            }
        }
#pragma unroll
        for (int m = 0; m < MG; ++m)
#pragma unroll
            for (int c = 0; c < NG; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r) sums[wave][m * NG + c][r][lane] = acc[m][c][r];
        __syncthreads();
        // the sum of row m, column c of the tile
        auto total = [&](int m, int c) {
            const int cell = m / 16 * NG + (TB ? c / 16 : c % NG), l = (TB ? c % 16 : c / NG) + 16 * (m % 16 / 4);
            float v = sums[0][cell][m & 3][l];
#pragma unroll
            for (int w = 1; w < kRowsWaves; ++w) v += sums[w][cell][m & 3][l];
            return v;
        };
        // Column c of the tile is column n of C; as stored, a lane that was moved back
        // has columns that its neighbours store.
        auto column = [&](int c) {
            if (TB) return n0 + c < p.N ? n0 + c : -1;
            const int wanted = n0 + c / NG * NG, n = min(wanted, p.N - NG) + c % NG;
            return wanted < p.N && n >= wanted ? n : -1;
        };
        if (p.mode != kStore) {
            // NG == 4: a wavefront a row
            for (int m = wave; m < 16 * MG && m < p.M; m += kRowsWaves) {
                const int n = lane < 16 * NG ? column(lane) : -1;
                const float v = n >= 0 ? total(m, lane) : -__builtin_inff();
                float top = v;
                for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
                float s = n >= 0 ? expf(v - (top == -__builtin_inff() ? 0.0f : top)) : 0.0f;
                for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
                if (lane == 0) p.stats[static_cast<int64_t>(m) * p.groups + n0 / 64] = stat2{top, s};
                if (n >= 0 && p.target[m] == n) p.at_target[m] = v;
                if (n >= 0 && p.mode == kStoreStats) p.c.p[m * p.c.ld + n] = v;
            }
        } else {
            for (int o = threadIdx.x; o < 256 * MG * NG; o += 64 * kRowsWaves) {
                const int c = o % (16 * NG), m = o / (16 * NG), n = column(c);
                if (m >= p.M || n < 0) continue;
                float z = total(m, c);
                if (p.splits > 1) {
                    p.slices[(slice * p.M + m) * p.N + n] = z;
                    continue;
                }
                if (p.e.bias.p != nullptr) z += p.e.bias.p[b * p.e.bias.stride + n];
                if (p.e.pre.p != nullptr) p.e.pre.p[b * p.e.pre.stride + m * p.e.pre.ld + n] = z;
                float v = activate(p.e.activation, z);
                if (p.e.residual.p != nullptr)
                    v += p.e.residual.p[b * p.e.residual.stride + m * p.e.residual.ld + n];
                p.c.p[b * p.c.stride + m * p.c.ld + n] = v;
            }
        }
        __syncthreads();
    }
}

template <int MG, int NG, bool TB>
hipError_t launch(const Product &p, hipStream_t stream) {
    const int tn = static_cast<int>(div_up(p.N, 16 * NG));
    const int64_t tiles = p.batch * p.splits * tn;
    const int len = static_cast<int>(div_up(div_up(p.K, 64), p.splits)) * 64;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20));
    rows_kernel<MG, NG, TB><<<grid, 64 * kRowsWaves, 0, stream>>>(p, tn, tiles, len);
    return hipGetLastError();
}

template <int NG>
hipError_t launch_columns(const Product &p, hipStream_t stream) {
    if (p.M <= 16) return p.tb ? launch<1, NG, true>(p, stream) : launch<1, NG, false>(p, stream);
    if (p.M <= 32) return p.tb ? launch<2, NG, true>(p, stream) : launch<2, NG, false>(p, stream);
    if (p.M <= 48) return p.tb ? launch<3, NG, true>(p, stream) : launch<3, NG, false>(p, stream);
    return p.tb ? launch<4, NG, true>(p, stream) : launch<4, NG, false>(p, stream);
}

}  // namespace

hipError_t launch_rows(const Product &p, int columns, hipStream_t stream) {
    return columns == 4 ? launch_columns<4>(p, stream)
           : columns == 2 ? launch_columns<2>(p, stream)
                          : launch_columns<1>(p, stream);
}

}  // namespace fused
}  // namespace gemm_f32_impl
