// The fused products that are small, or have few rows of op(A), so that reading B is
// the work.

#include <type_traits>

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {
namespace {

// The epilogue for one sum, or its slice.
__device__ __forceinline__ void finish(const Product &p, int64_t b, int64_t slice, int m, int n, float z) {
    if (p.splits > 1) {
        p.slices[(slice * p.M + m) * p.N + n] = z;
        return;
    }
    if (p.mode == kStoreSome && p.target[m] == p.ignore) z = 0.0f;
    if (p.e.bias.p != nullptr) z += p.e.bias.p[b * p.e.bias.stride + n];
    if (p.e.pre.p != nullptr) p.e.pre.p[b * p.e.pre.stride + m * p.e.pre.ld + n] = z;
    float v = activate(p.e.activation, z);
    if (p.e.residual.p != nullptr) v += p.e.residual.p[b * p.e.residual.stride + m * p.e.residual.ld + n];
    p.c.p[b * p.c.stride + m * p.c.ld + n] = v;
}

// One sum of 16 neighbouring columns that 16 lanes hold, all of which come here
// together; `in`: it is one of C.
__device__ __forceinline__ void store_cell(const Product &p, int64_t b, int64_t slice, int m, int n, float v, bool in) {
    if (p.mode < kStats) {
        if (in) finish(p, b, slice, m, n, v);
        return;
    }
    const float top = over_lanes<16>(in ? v : -__builtin_inff(), [](float a, float b) { return fmaxf(a, b); });
    const float s = over_lanes<16>(in ? quick_exp(v - base_of(top)) : 0.0f,
                                   [](float a, float b) { return a + b; });
    if (!in) return;
    if (n % 16 == 0) p.stats[static_cast<int64_t>(m) * p.groups + n / 16] = stat2{top, s};
    if (p.target[m] == n) p.at_target[m] = v;
    if (p.mode == kStoreStats) p.c.p[m * p.c.ld + n] = v;
}

// Small products and few rows, on FP32 multiplies straight from global memory: a
// workgroup of 8 wavefronts holds 16 MG rows and 16 NG columns; its wavefronts
// take steps of 64 (32) k in turn, a step ahead, and their sums are added in LDS
// in a fixed order.  In v_mfma_f32_16x16x4_f32 lane l holds one k, l / 16, of
// row (column) l % 16; here lane group g = l / 16 holds k 16 u + 4 g + j of a step in
// instruction (u, j).  So where k is contiguous a lane's part of a row is 16
// bytes; where rows are, it takes MG (NG) neighbours at every k.  A launch, one chain
// of loads and the joining of 8 sums bound it at small sizes (both products of a
// 256 x 256 x 256 gradient 4.7 us, the 64 x 1000 x 256 logits of a loss 5.2), memory at few rows (16 x 4096 x
// 4096, B transposed, 18 us, 3.7 TB/s).
constexpr int kRowsWaves = 8;
constexpr int quads_of(int mg, int ng) { return (mg + ng) * 4 <= 20 ? 4 : 2; }  // for two steps' registers

// One operand's share of a lane: G groups of 16 rows.
template <int G, bool KC>
struct Lines {
    typedef float group_t __attribute__((ext_vector_type(G < 2 ? 2 : G), aligned(4)));
    const float *p[KC ? G : 1];
    int64_t ld;
    // rows past the end repeat the last ones' and are not stored
    __device__ __forceinline__ Lines(const Operand &x, int64_t batch, int first, int rows, int at) {
        ld = x.ld;
        const float *base = x.p + batch * x.stride;
        if constexpr (KC) {
#pragma unroll
            for (int g = 0; g < G; ++g) p[g] = base + static_cast<int64_t>(min(first + 16 * g + at, rows - 1)) * ld;
        } else {
            p[0] = base + min(first + G * at, rows - G);  // moved back from past the end
        }
    }
    // Row r of the tile: its group, its place among 16, the row of the operand.
    static __device__ __forceinline__ int group(int r) { return KC ? r / 16 : r % G; }
    static __device__ __forceinline__ int place(int r) { return KC ? r % 16 : r / G; }
    // -1: past the end, or a neighbour's where the lane was moved back
    static __device__ __forceinline__ int row(int first, int r, int rows) {
        const int wanted = KC ? first + r : first + r / G * G, got = KC ? wanted : min(wanted, rows - G) + r % G;
        return wanted < rows && got >= wanted ? got : -1;
    }
    // 4 k from k on; past k1, if not WHOLE, zero, and, if SKIP, where skip[k] is `ignore`.
    template <bool WHOLE, bool SKIP>
    __device__ __forceinline__ void load(int k, int k1, f32x4 (&v)[G], const int64_t *skip, int64_t ignore) const {
        if constexpr (KC) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if constexpr (WHOLE) {
                    v[g] = *reinterpret_cast<const float4u *>(p[g] + k);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[g][j] = k + j < k1 ? p[g][k + j] : 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bool in = WHOLE || k + j < k1;
                const int64_t at = in ? k + j : k1 - 1;
                const float *from = p[0] + at * ld;
                if constexpr (SKIP) in = in && skip[at] != ignore;
                if constexpr (G == 1) {
                    v[0][j] = in ? *from : 0.0f;
                } else {
                    const group_t x = *reinterpret_cast<const group_t *>(from);
#pragma unroll
                    for (int g = 0; g < G; ++g) v[g][j] = in ? x[g] : 0.0f;
                }
            }
        }
    }
};

// How a product is laid out over workgroups.
struct Grid {
    int tiles_m, tiles_n, len, shape;  // k a slice
    int64_t tiles;
};
constexpr int sums_bytes(int mg, int ng) { return kRowsWaves * mg * ng * 4 * 64 * 4; }

// Tile t.
template <int MG, int NG, bool TA, bool TB, bool SKIP>
__device__ __forceinline__ void rows_tile(const Product &p, const Grid &g, int64_t t, float *memory) {
    constexpr int kQuads = quads_of(MG, NG), kStep = 16 * kQuads;
    using LA = Lines<MG, !TA>;
    using LB = Lines<NG, TB>;
    auto sums = reinterpret_cast<float(*)[MG * NG][4][64]>(memory);
    const int lane = threadIdx.x & 63, at = lane & 15, group = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t per = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
    const int64_t slice = t / per, b = slice / p.splits;
    int tm, tn;
    grouped_tile(static_cast<int>(t - slice * per), g.tiles_m, g.tiles_n, 8, tm, tn);
    const int m0 = tm * 16 * MG, n0 = tn * 16 * NG;
    const int k0 = static_cast<int>(slice - b * p.splits) * g.len;
    const int k1 = max(k0, static_cast<int>(min(static_cast<int64_t>(k0) + g.len, static_cast<int64_t>(p.K))));
    const LA la(p.a, b, m0, p.M, at);
    const LB lb(p.b, b, n0, p.N, at);
    struct Step {
        f32x4 a[kQuads][MG], b[kQuads][NG];
    };
    auto load = [&](int s, auto whole_) {
        constexpr bool kWhole = decltype(whole_)::value;
        Step x;
#pragma unroll
        for (int u = 0; u < kQuads; ++u) {
            const int k = k0 + s * kStep + 16 * u + 4 * group;
            lb.template load<kWhole, SKIP>(k, k1, x.b[u], p.target_k, p.ignore);
            la.template load<kWhole, false>(k, k1, x.a[u], nullptr, 0);
        }
        return x;
    };
    f32x4 acc[MG][NG];
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
        for (int c = 0; c < NG; ++c) acc[m][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto step = [&](const Step &x) {
#pragma unroll
        for (int u = 0; u < kQuads; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int m = 0; m < MG; ++m)
#pragma unroll
                    for (int c = 0; c < NG; ++c)
                        acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(x.a[u][m][j], x.b[u][c][j], acc[m][c], 0, 0, 0);
    };
    constexpr std::true_type all;
    const int whole = (k1 - k0) / kStep;
    if (wave < whole) {
        // loads past the last step repeat it and are not used: what is on its
        // way is known at every point
        const int count = (whole - wave + kRowsWaves - 1) / kRowsWaves;
        // Where rows are a power of two apart, workgroups that all start at
        // k0 ask the same few memory channels: each starts elsewhere.
        const int turn = TB && NG == 1 ? static_cast<int>(t % count) : 0;
        auto turned = [&](int s) {
            s = min(s, count - 1) + turn;
            return wave + (s < count ? s : s - count) * kRowsWaves;
        };
        Step x = load(turned(0), all), y;
        int s = 0;
        for (; s + 1 < count; s += 2) {
            y = load(turned(s + 1), all);
            step(x);
            x = load(turned(s + 2), all);
            step(y);
        }
        if (s < count) step(x);
    }
    if (whole * kStep < k1 - k0 && whole % kRowsWaves == wave) step(load(whole, std::false_type{}));
#pragma unroll
    for (int m = 0; m < MG; ++m)
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[wave][m * NG + c][r][lane] = acc[m][c][r];
    __syncthreads();
    for (int o = threadIdx.x; o < 256 * MG * NG; o += 64 * kRowsWaves) {
        const int c = o % (16 * NG), r = o / (16 * NG), q = LA::place(r);
        const int cell = LA::group(r) * NG + LB::group(c), l = LB::place(c) + 16 * (q / 4);
        float v = sums[0][cell][q & 3][l];
#pragma unroll
        for (int w = 1; w < kRowsWaves; ++w) v += sums[w][cell][q & 3][l];
        const int m = LA::row(m0, r, p.M), n = LB::row(n0, c, p.N);
        store_cell(p, b, slice, m, n, v, m >= 0 && n >= 0);
    }
    __syncthreads();
}

template <int MG, int NG, bool TA, bool TB, bool SKIP>
__global__ __launch_bounds__(64 * kRowsWaves) void rows_kernel(Product p, Grid g) {
    __shared__ __align__(16) float memory[sums_bytes(MG, NG) / 4];
    for (int64_t t = xcd_remap(blockIdx.x, gridDim.x); t < g.tiles; t += gridDim.x)
        rows_tile<MG, NG, TA, TB, SKIP>(p, g, t, memory);
}

// Two small products in one launch, as a gradient has them: neither has to wait
// for the other, and a launch takes as long as one of them.
template <bool TA, bool TB, bool SKIP>
__device__ __forceinline__ void any_shape(const Product &p, const Grid &g, int64_t t, float *memory) {
    if (g.shape == 16 + 1)
        rows_tile<1, 1, TA, TB, SKIP>(p, g, t, memory);
    else if (g.shape == 16 + 2)
        rows_tile<1, 2, TA, TB, SKIP>(p, g, t, memory);
    else
        rows_tile<2, 2, TA, TB, SKIP>(p, g, t, memory);
}
template <bool TA1, bool TB1, bool TA2, bool TB2, bool SKIP2>
__global__ __launch_bounds__(64 * kRowsWaves) void pair_kernel(Product p, Grid g, Product q, Grid h) {
    __shared__ __align__(16) float memory[sums_bytes(2, 2) / 4];
    const int first = static_cast<int>(g.tiles), t = static_cast<int>(blockIdx.x);
    if (t < first)
        any_shape<TA1, TB1, false>(p, g, xcd_remap(t, first), memory);
    else
        any_shape<TA2, TB2, SKIP2>(q, h, xcd_remap(t - first, static_cast<int>(h.tiles)), memory);
}

// B stored N x K, MR (1, 2 or 4) rows of op(A): a wavefront holds 4 columns,
// which are rows of B that it reads 1 KiB at a time, and a lane the products of
// its 4 k; a workgroup of 4 wavefronts 16 columns.  The 64 lanes' sums are added by halves.
// Memory bounds it: 1 x 14336 x 4096 36 to 42 us by card (5.6 to 6.5 TB/s; a copy reaches
// 5.2), 1 x 32768 x 4096 86 (6.2).
template <int MR, bool TA>
__global__ __launch_bounds__(256) void vector_kernel(Product p, int tiles_n, int64_t tiles, int len) {
    constexpr int R = 4, kStep = 256, U = 2;  // U steps' loads on their way at once
    __shared__ float cells[MR][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t slice = t / tiles_n, b = slice / p.splits;
        const int n0 = static_cast<int>(t - slice * tiles_n) * 16;
        const int k0 = static_cast<int>(slice - b * p.splits) * len;
        const int k1 = max(k0, static_cast<int>(min(static_cast<int64_t>(k0) + len, static_cast<int64_t>(p.K))));
        const float *A = p.a.p + b * p.a.stride, *B = p.b.p + b * p.b.stride;
        // rows and columns past the end repeat the last ones' and are not stored
        const float *row[R], *x[MR];
#pragma unroll
        for (int r = 0; r < R; ++r) row[r] = B + static_cast<int64_t>(min(n0 + R * wave + r, p.N - 1)) * p.b.ld;
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const int64_t q = min(m, p.M - 1);
            x[m] = A + (TA ? q : q * p.a.ld);
        }
        float acc[MR][R];
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[m][r] = 0.0f;
        struct Step {
            f32x4 w[R], v[MR];
        };
        auto load = [&](int s) {
            const int k = k0 + s * kStep + 4 * lane;
            Step q;
#pragma unroll
            for (int r = 0; r < R; ++r) q.w[r] = *reinterpret_cast<const float4u *>(row[r] + k);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                if constexpr (!TA) {
                    q.v[m] = *reinterpret_cast<const float4u *>(x[m] + k);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q.v[m][e] = x[m][(k + e) * p.a.ld];
                }
            }
            return q;
        };
        auto use = [&](const Step &q) {
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][r] = fmaf(q.v[m][e], q.w[r][e], acc[m][r]);
        };
        const int whole = (k1 - k0) / kStep;
        if (whole > 0) {
            // loads past the last step repeat it and are not used: what is on its
            // way is known at every point
            // Where rows are a power of two apart, wavefronts that all start
            // at k0 ask the same few memory channels: each starts elsewhere.
            const int turn = static_cast<int>((t * 4 + wave) % whole);
            auto turned = [&](int s) {
                s = min(s, whole - 1) + turn;
                return s < whole ? s : s - whole;
            };
            Step q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = load(turned(u));
            int s = 0;
            for (; s + U <= whole; s += U)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    use(q[u]);
                    q[u] = load(turned(s + U + u));
                }
#pragma unroll
            for (int u = 0; u < U - 1; ++u)
                if (s + u < whole) use(q[u]);
        }
        for (int k = k0 + whole * kStep + lane; k < k1; k += 64)  // what is left of K
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const float v = x[m][TA ? k * p.a.ld : k];
#pragma unroll
                for (int r = 0; r < R; ++r) acc[m][r] = fmaf(v, row[r][k], acc[m][r]);
            }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                for (int d = 32; d > 0; d /= 2) acc[m][r] += __shfl_xor(acc[m][r], d);
                if (lane == 0) cells[m][R * wave + r] = acc[m][r];
            }
        __syncthreads();
        const int m = threadIdx.x / 16, n = n0 + threadIdx.x % 16;
        if (m < MR) {
            const float v = cells[m][threadIdx.x % 16];
            store_cell(p, b, slice, m, n, v, m < p.M && n < p.N);
        }
        __syncthreads();
    }
}

template <int MR, bool TA>
hipError_t launch_vector(const Product &p, hipStream_t stream) {
    const int tn = static_cast<int>(div_up(p.N, 16));
    const int64_t tiles = p.batch * p.splits * tn;
    const int len = static_cast<int>(div_up(div_up(p.K, 256), p.splits)) * 256;
    vector_kernel<MR, TA><<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20)), 256, 0, stream>>>(p, tn, tiles, len);
    return hipGetLastError();
}

Grid grid_of(const Product &p, int shape) {
    const int mg = shape >> 4, ng = shape & 15;
    Grid g{};
    g.tiles_m = static_cast<int>(div_up(p.M, 16 * mg)), g.tiles_n = static_cast<int>(div_up(p.N, 16 * ng));
    g.tiles = p.batch * p.splits * g.tiles_m * g.tiles_n;
    g.len = static_cast<int>(div_up(div_up(p.K, 64), p.splits)) * 64;
    g.shape = shape;
    return g;
}

template <int MG, int NG, bool TA, bool TB, bool SKIP = false>
hipError_t launch(const Product &p, hipStream_t stream) {
    const Grid g = grid_of(p, 16 * MG + NG);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(g.tiles, 1 << 20));
    rows_kernel<MG, NG, TA, TB, SKIP><<<grid, 64 * kRowsWaves, 0, stream>>>(p, g);
    return hipGetLastError();
}

template <int MG, int NG>
hipError_t launch_form(const Product &p, hipStream_t stream) {
    if (p.target_k != nullptr) return launch<MG, NG, true, false, true>(p, stream);
    return p.ta ? (p.tb ? launch<MG, NG, true, true>(p, stream) : launch<MG, NG, true, false>(p, stream))
                : (p.tb ? launch<MG, NG, false, true>(p, stream) : launch<MG, NG, false, false>(p, stream));
}

}  // namespace

hipError_t launch_rows(const Product &p, int shape, hipStream_t stream) {
    if (shape == 0)
        return p.M == 1   ? (p.ta ? launch_vector<1, true>(p, stream) : launch_vector<1, false>(p, stream))
               : p.M == 2 ? (p.ta ? launch_vector<2, true>(p, stream) : launch_vector<2, false>(p, stream))
                          : (p.ta ? launch_vector<4, true>(p, stream) : launch_vector<4, false>(p, stream));
    switch (shape) {
        case 16 + 1: return launch_form<1, 1>(p, stream);
        case 16 + 2: return launch_form<1, 2>(p, stream);
        case 16 + 4: return launch_form<1, 4>(p, stream);
        case 32 + 1: return launch_form<2, 1>(p, stream);
        case 32 + 2: return launch_form<2, 2>(p, stream);
        case 32 + 4: return launch_form<2, 4>(p, stream);
        case 64 + 2: return launch_form<4, 2>(p, stream);
        default: return hipErrorInvalidConfiguration;
    }
}

bool launch_rows_pair(const Product &p, int shape_p, const Product &q, int shape_q, hipStream_t stream, hipError_t *err) {
    auto taken = [](int shape) { return shape == 16 + 1 || shape == 16 + 2 || shape == 32 + 2; };
    if (!taken(shape_p) || !taken(shape_q) || p.splits > 1 || q.splits > 1 || p.target_k != nullptr) return false;
    const Grid g = grid_of(p, shape_p), h = grid_of(q, shape_q);
    if (g.tiles + h.tiles > 1 << 20) return false;
    const unsigned grid = static_cast<unsigned>(g.tiles + h.tiles), threads = 64 * kRowsWaves;
    const int form = p.ta * 8 + p.tb * 4 + q.ta * 2 + q.tb;
    if (q.target_k != nullptr) {
        if (form != 2) return false;
        pair_kernel<false, false, true, false, true><<<grid, threads, 0, stream>>>(p, g, q, h);
    } else {
        switch (form) {  // of gemm_f32_fused_grad's two products, by opA and opB
            case 4 + 2: pair_kernel<false, true, true, false, false><<<grid, threads, 0, stream>>>(p, g, q, h); break;
            case 2: pair_kernel<false, false, true, false, false><<<grid, threads, 0, stream>>>(p, g, q, h); break;
            case 4: pair_kernel<false, true, false, false, false><<<grid, threads, 0, stream>>>(p, g, q, h); break;
            case 8 + 4 + 2 + 1: pair_kernel<true, true, true, true, false><<<grid, threads, 0, stream>>>(p, g, q, h); break;
            default: return false;
        }
    }
    *err = hipGetLastError();
    return true;
}

}  // namespace fused
}  // namespace gemm_f32_impl
