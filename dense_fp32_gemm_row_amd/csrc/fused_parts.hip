// What stands beside the fused tile kernels: the sum of slices, the slope of
// a layer's activation with its bias gradient, and the rest of the cross
// entropy.  All of it reads and writes its matrices once, by memory's rate.

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {
namespace {

// 4 neighbours of a row, of which `left` are inside it.
__device__ __forceinline__ f32x4 read4(const float *p, int64_t left) {
    f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
    if (left >= 4) {
        v = *reinterpret_cast<const float4u *>(p);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) v[e] = p[e];
    }
    return v;
}
__device__ __forceinline__ void write4(float *p, int64_t left, f32x4 v) {
    if (left >= 4) {
        *reinterpret_cast<float4u *>(p) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) p[e] = v[e];
    }
}

// C = epilogue(sum of slices), 4 neighbours of a row a thread, slices in order: 1000 x
// 1023 in two slices 5 us, most of it a launch (an element a thread, 64-bit divisions: 6.5).
// SOME: kStoreSome (a branch for it in every product's sum: 6.8 -> 7.6 us for two).
template <bool SOME>
__device__ __forceinline__ void sum_slices(const Product &p, int64_t block, int64_t blocks) {
    const int64_t per = static_cast<int64_t>(p.M) * p.N, rows = p.batch * p.M;
    const unsigned strips = (static_cast<unsigned>(p.N) + 3) / 4;
    for (int64_t o = block * 256; o < rows * strips; o += blocks * 256) {
        const int64_t first = o / strips;  // the workgroup's first row: of all, by 64 bits, the others by 32
        const unsigned at = static_cast<unsigned>(o - first * strips) + threadIdx.x;
        const int64_t row = first + at / strips;
        if (row >= rows) break;
        const int64_t b = p.batch == 1 ? 0 : row / p.M, m = row - b * p.M, n = 4 * static_cast<int64_t>(at % strips);
        const int64_t left = p.N - n;
        const float *W = p.slices + b * p.splits * per + m * p.N + n;
        f32x4 z = read4(W, left);
#pragma unroll 4
        for (int s = 1; s < p.splits; ++s) z += read4(W + s * per, left);
        if constexpr (SOME)
            if (p.target[m] == p.ignore) z = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (p.e.bias.p != nullptr) z += read4(p.e.bias.p + b * p.e.bias.stride + n, left);
        if (p.e.pre.p != nullptr) write4(p.e.pre.p + b * p.e.pre.stride + m * p.e.pre.ld + n, left, z);
        if (p.e.activation != GEMM_F32_ACT_NONE)
#pragma unroll 1
            for (int e = 0; e < 4; ++e) z = f32x4{z[1], z[2], z[3], activate(p.e.activation, z[0])};
        if (p.e.residual.p != nullptr) z += read4(p.e.residual.p + b * p.e.residual.stride + m * p.e.residual.ld + n, left);
        write4(p.c.p + b * p.c.stride + m * p.c.ld + n, left, z);
    }
}
template <bool SOME>
__global__ __launch_bounds__(256) void sum_slices_kernel(Product p) {
    sum_slices<SOME>(p, blockIdx.x, gridDim.x);
}
// Workgroups 0 .. first - 1 take p.
template <bool SOME>
__global__ __launch_bounds__(256) void sum_two_kernel(Product p, Product q, unsigned first) {
    if (blockIdx.x < first)
        sum_slices<SOME>(p, blockIdx.x, first);
    else
        sum_slices<false>(q, blockIdx.x - first, gridDim.x - first);
}

// A block of rows of 4 LANES columns, 4 a lane, its rows shared by WAVES wavefronts and
// the 64 / LANES parts of each: dZ, and the columns' sums over the block.  Memory bounds it
// (4096 x 4096, GELU, 41 us, 4.9 TB/s), at 256 x 256 one chain of loads and sums in 4
// workgroups (8.5 us, with the bias gradient, which has no launch of its own there).
template <int KIND, int WAVES, int LANES>
__global__ __launch_bounds__(64 * WAVES) void slope_kernel(Slope s, int64_t strips, int64_t units) {
    constexpr int kParts = 64 * WAVES / LANES;
    __shared__ f32x4 sums[kParts][LANES];
    const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t strip = u % strips, rest = u / strips, block = rest % s.blocks, b = rest / s.blocks;
        const int64_t n = strip * (4 * LANES) + 4 * lane, left = s.N - n;
        const int64_t first = block * s.rows, last = min(first + s.rows, int64_t{s.M});
        const float *dc = s.dc.p + b * s.dc.stride + n, *pre = s.pre.p + b * s.pre.stride + n;
        float *dz = s.dz.p + b * s.dz.stride + n;
        f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
        if (left > 0) {
#pragma unroll 4
            for (int64_t m = first + part; m < last; m += kParts) {
                f32x4 v = read4(dc + m * s.dc.ld, left);
                if constexpr (KIND != GEMM_F32_ACT_NONE) {
                    const f32x4 z = read4(pre + m * s.pre.ld, left);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] *= slope(KIND, z[e]);
                }
                if (s.dz.p != nullptr) write4(dz + m * s.dz.ld, left, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += v[e];
            }
        }
        if (s.dbias.p == nullptr) continue;
        sums[part][lane] = sum;
        __syncthreads();
        if (part == 0 && left > 0) {
#pragma unroll
            for (int w = 1; w < kParts; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += sums[w][lane][e];
            write4(s.blocks == 1 ? s.dbias.p + b * s.dbias.stride + n : s.partial + (b * s.blocks + block) * s.N + n, left,
                   sum);
        }
        __syncthreads();
    }
}

// The blocks' sums of 16 columns, shared by 16 threads a column (64 blocks of 4096
// columns 4.9 us, a launch's time).
__global__ __launch_bounds__(256) void bias_kernel(Slope s, int64_t strips, int64_t units) {
    __shared__ float sums[16][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t b = u / strips, n = (u - b * strips) * 16 + c;
        const float *from = s.partial + b * s.blocks * s.N + n;
        float sum = 0.0f;
        if (n < s.N)
#pragma unroll 4
            for (int q = part; q < s.blocks; q += 16) sum += from[static_cast<int64_t>(q) * s.N];
        sums[part][c] = sum;
        __syncthreads();
        if (part == 0 && n < s.N) {
            for (int q = 1; q < 16; ++q) sum += sums[q][c];
            s.dbias.p[b * s.dbias.stride + n] = sum;
        }
        __syncthreads();
    }
}

// exp(logit - lse) - (v == target), times g.
__device__ __forceinline__ float gradient(const Loss &l, float x, float lse, float g, int64_t v, int64_t target) {
    const float p = g * (quick_exp(x - lse) - (v == target ? 1.0f : 0.0f));
    return target == l.ignore ? 0.0f : target >= 0 && target < l.V ? p : __builtin_nanf("");
}

// A workgroup a row: its pieces' statistics joined, in a fixed order (2048 rows of 512
// pieces 5.6 us, a launch's time); with GRAD the row's gradient, too, which saves a launch where there
// are few logits (64 x 1000 5.8 us).
template <bool GRAD>
__global__ __launch_bounds__(256) void loss_kernel(Loss l) {
    __shared__ float tops[4], sums[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < l.T; t += gridDim.x) {
        float m = -__builtin_inff(), s = 0.0f;
#pragma unroll 4
        for (int g = threadIdx.x; g < l.groups; g += 256) {
            const stat2 q = l.stats[t * l.groups + g];
            merge_stats(m, s, q.x, q.y);
        }
        for (int d = 1; d < 64; d *= 2) {
            const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
            merge_stats(m, s, m2, s2);
        }
        if (lane == 0) tops[wave] = m, sums[wave] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w) merge_stats(m, s, tops[w], sums[w]);
            const float lse = m + logf(s);
            l.lse[t] = lse;
            if (l.loss != nullptr) {
                const int64_t target = l.target[t];
                l.loss[t] = target == l.ignore ? 0.0f
                            : target >= 0 && target < l.V ? lse - l.at_target[t] : __builtin_nanf("");
            }
            if constexpr (GRAD) tops[0] = lse;
        }
        __syncthreads();
        if constexpr (GRAD) {
            const float lse = tops[0], g = l.grad_loss != nullptr ? l.grad_loss[t] : 1.0f;
            const int64_t target = l.target[t];
            float *row = l.logits + t * l.ld;
#pragma unroll 4
            for (int64_t v = threadIdx.x; v < l.V; v += 256) row[v] = gradient(l, row[v], lse, g, v, target);
            __syncthreads();
        }
    }
}

// `rows` rows of 1024 columns, 4 a thread (4096 x 131072 841 us, 5.1 TB/s, a copy's rate;
// 517 x 32003 28).
__global__ __launch_bounds__(256) void probabilities_kernel(Loss l, int64_t strips, int64_t units, int rows) {
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t block = u / strips, v = (u - block * strips) * 1024 + 4 * threadIdx.x, left = l.V - v;
        if (left <= 0) continue;
        const int64_t first = block * rows, last = min(first + rows, static_cast<int64_t>(l.T));
        constexpr int kAtOnce = 4;
        for (int64_t t0 = first; t0 < last; t0 += kAtOnce) {
            f32x4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) x[i] = read4(l.logits + min(t0 + i, last - 1) * l.ld + v, left);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int64_t t = t0 + i;
                if (t >= last) break;
                const int64_t target = l.target[t];
                const float lse = l.lse[t], g = l.grad_loss != nullptr ? l.grad_loss[t] : 1.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = gradient(l, x[i][e], lse, g, v + e, target);
                write4(l.logits + t * l.ld + v, left, x[i]);
            }
        }
    }
}

__device__ __forceinline__ void count(RowStat &s, float x) {
    const int bits = __builtin_bit_cast(int, x) & 0x7fffffff, e = bits >> 23;
    s.top = max(s.top, e);
    // a value below 2^-126 has up to 23 leading zeros in its place
    s.count += bits != 0, s.sum += bits == 0 ? 0 : e == 0 ? -23 : e;
}
__device__ __forceinline__ void join(RowStat &s, int top, int n, int sum) {
    s.top = max(s.top, top), s.count += n, s.sum += sum;
}

// One operand, `rows` rows of each of `batch` matrices, k in `blocks` blocks of `len`.
struct StatJob {
    Operand x;
    bool kc;
    int rows, K, blocks, len;
    RowStat *out;
    int64_t strips, units;  // workgroups: [batch][block][strip]
};

// Where k is contiguous a wavefront takes a row's block, else a workgroup 256
// rows' (a row a thread).  Memory bounds it: two operands of 4096 x 4096 26 us (5.2 TB/s),
// 131072 x 2048 by columns 229 (4.7).
__global__ __launch_bounds__(256) void row_stats_kernel(StatJob a, StatJob b, int64_t batch) {
    const int tid = threadIdx.x, lane = tid & 63;
    for (int64_t u = blockIdx.x; u < a.units + b.units; u += gridDim.x) {
        const bool second = u >= a.units;
        const StatJob &j = second ? b : a;
        const int64_t w = second ? u - a.units : u, strip = w % j.strips, rest = w / j.strips;
        const int block = static_cast<int>(rest % j.blocks);
        const int64_t n = rest / j.blocks;
        const int64_t k0 = static_cast<int64_t>(block) * j.len, k1 = min(k0 + j.len, static_cast<int64_t>(j.K));
        const float *p = j.x.p + n * j.x.stride;
        RowStat s{0, 0, 0, 0};
        int64_t row;
        if (j.kc) {
            row = strip * 4 + (tid >> 6);
            if (row >= j.rows) continue;
            p += row * j.x.ld;
            // four at once; loads past the end repeat the last one's and do not count
            const int64_t k4 = k1 - 4;
            if (k4 >= k0)
                for (int64_t k = k0 + 4 * lane; k - 4 * lane <= k4; k += 1024) {
                    f32x4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4u *>(p + min(k + 256 * i, k4));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) count(s, k + 256 * i <= k4 ? v[i][e] : 0.0f);
                }
            const int64_t rest = k0 + (k1 - k0) / 4 * 4 + lane;
            if (rest < k1) count(s, p[rest]);  // the last three at most
            for (int d = 1; d < 64; d *= 2) join(s, __shfl_xor(s.top, d), __shfl_xor(s.count, d), __shfl_xor(s.sum, d));
            if (lane != 0) continue;
        } else {
            row = strip * 256 + tid;
            if (row >= j.rows) continue;
            p += row;
#pragma unroll 16
            for (int64_t k = k0; k < k1; ++k) count(s, p[k * j.x.ld]);
        }
        j.out[(block * batch + n) * j.rows + row] = s;
    }
}

unsigned blocks_for(int64_t n) { return static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(n, 1), 1 << 21)); }

}  // namespace

static unsigned sum_blocks(const Product &p) { return blocks_for(div_up(p.batch * p.M * div_up(p.N, 4), 256)); }

hipError_t launch_sum_slices(const Product &p, hipStream_t stream) {
    if (p.mode == kStoreSome)
        sum_slices_kernel<true><<<sum_blocks(p), 256, 0, stream>>>(p);
    else
        sum_slices_kernel<false><<<sum_blocks(p), 256, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_sum_slices(const Product &p, const Product &q, hipStream_t stream) {
    const unsigned first = sum_blocks(p);
    if (p.mode == kStoreSome)
        sum_two_kernel<true><<<first + sum_blocks(q), 256, 0, stream>>>(p, q, first);
    else
        sum_two_kernel<false><<<first + sum_blocks(q), 256, 0, stream>>>(p, q, first);
    return hipGetLastError();
}

template <int WAVES, int LANES>
static void run_slope(const Slope &s, hipStream_t stream) {
    const int64_t strips = div_up(s.N, 4 * LANES), units = strips * s.blocks * s.batch;
    const unsigned grid = blocks_for(units), threads = 64 * WAVES;
    switch (s.activation) {
        case GEMM_F32_ACT_RELU: slope_kernel<GEMM_F32_ACT_RELU, WAVES, LANES><<<grid, threads, 0, stream>>>(s, strips, units); break;
        case GEMM_F32_ACT_GELU: slope_kernel<GEMM_F32_ACT_GELU, WAVES, LANES><<<grid, threads, 0, stream>>>(s, strips, units); break;
        case GEMM_F32_ACT_GELU_TANH:
            slope_kernel<GEMM_F32_ACT_GELU_TANH, WAVES, LANES><<<grid, threads, 0, stream>>>(s, strips, units);
            break;
        case GEMM_F32_ACT_SILU: slope_kernel<GEMM_F32_ACT_SILU, WAVES, LANES><<<grid, threads, 0, stream>>>(s, strips, units); break;
        default: slope_kernel<GEMM_F32_ACT_NONE, WAVES, LANES><<<grid, threads, 0, stream>>>(s, strips, units);
    }
}

hipError_t launch_slope(const Slope &s, hipStream_t stream) {
    // One block of rows: dbias is its sum, 16 parts of a workgroup share it.
    if (s.blocks == 1)
        run_slope<4, 16>(s, stream);
    else
        run_slope<4, 64>(s, stream);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && s.dbias.p != nullptr && s.blocks != 1) {
        const int64_t lines = div_up(s.N, 16);
        bias_kernel<<<blocks_for(lines * s.batch), 256, 0, stream>>>(s, lines, lines * s.batch);
        err = hipGetLastError();
    }
    return err;
}

hipError_t launch_loss(const Loss &l, hipStream_t stream) {
    loss_kernel<false><<<blocks_for(l.T), 256, 0, stream>>>(l);
    return hipGetLastError();
}

hipError_t launch_loss_and_probabilities(const Loss &l, hipStream_t stream) {
    loss_kernel<true><<<blocks_for(l.T), 256, 0, stream>>>(l);
    return hipGetLastError();
}

hipError_t launch_probabilities(const Loss &l, hipStream_t stream) {
    const int64_t strips = div_up(l.V, 1024);
    // as many rows a workgroup as leave enough of them
    const int rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, l.T * strips / 1024)));
    const int64_t units = strips * div_up(l.T, rows);
    probabilities_kernel<<<blocks_for(units), 256, 0, stream>>>(l, strips, units, rows);
    return hipGetLastError();
}

namespace {
// The tiles' loads count bytes from a tile's first element in 32 bits: 256 rows
// of k, or 16 k of rows.
bool narrow_operand(int64_t ld, bool k_contiguous) {
    return k_contiguous ? ld <= (int64_t{1} << 22) - 64 : ld <= int64_t{1} << 25;
}
}  // namespace

hipError_t launch_row_stats(const Product &p, hipStream_t stream) {
    auto job = [&](const Operand &x, bool kc, int rows, int blocks, const RowStat *out) {
        StatJob j{x, kc, rows, p.K, blocks, static_cast<int>(div_up(p.K, blocks)), const_cast<RowStat *>(out), 0, 0};
        j.strips = div_up(rows, kc ? 4 : 256);
        j.units = j.strips * blocks * p.batch;
        return j;
    };
    const StatJob a = job(p.a, !p.ta, p.M, p.blocks_a, p.row_a), b = job(p.b, p.tb, p.N, p.blocks_b, p.row_b);
    row_stats_kernel<<<blocks_for(a.units + b.units), 256, 0, stream>>>(a, b, p.batch);
    return hipGetLastError();
}

namespace {
bool narrow(const Product &p) { return narrow_operand(p.a.ld, !p.ta) && narrow_operand(p.b.ld, p.tb); }
// (at most 2^61)
int64_t slices_bytes(const Choice &c, int64_t batch, int64_t M, int64_t N) {
    const __int128 n = c.splits > 1 ? static_cast<__int128>(4 * c.splits) * batch * M * N : 0;
    return static_cast<int64_t>(std::min<__int128>(n, __int128{1} << 61));
}
// Whether two products go into one launch of tiles: each as it would be by itself, so
// that its values are those, too.  (1000 x 777 x 1023 and 777 x 1023 x 1000, 224 workgroups each,
// 24 and 26 us and 6 each for their slices; together 34 and 7.)
bool paired(const Choice &c, const Choice &d, bool ta, bool tc, bool td) {
    return c.tile == d.tile && (c.tile == 1 || c.tile == 2) && !c.half && !d.half && !ta && tc && !td;
}
}  // namespace

namespace {
int64_t choice_space(const Choice &c, int64_t batch, int64_t M, int64_t N, int64_t K) {
    // either form of either operand
    const __int128 stats = c.half ? static_cast<__int128>(sizeof(RowStat)) * batch *
                                        (std::max(stat_blocks(M, K, true), stat_blocks(M, K, false)) * M +
                                         std::max(stat_blocks(N, K, true), stat_blocks(N, K, false)) * N)
                                  : 0;
    return static_cast<int64_t>(std::min<__int128>(slices_bytes(c, batch, M, N) + stats, __int128{1} << 61));
}
Choice choice_of(const Product &p) {
    return choose(p.tb, p.batch, p.M, p.N, p.K, p.space != nullptr, p.use);
}
}  // namespace

int64_t product_space(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, Use use) {
    return choice_space(choose(tb, batch, M, N, K, true, use), batch, M, N, K);
}

int64_t two_space(const Sizes &p, const Sizes &q) {
    const Choice c = choose(p.tb, p.batch, p.M, p.N, p.K, true, p.use), d = choose(q.tb, q.batch, q.M, q.N, q.K, true, q.use);
    const int64_t m = choice_space(c, p.batch, p.M, p.N, p.K), n = choice_space(d, q.batch, q.M, q.N, q.K);
    return paired(c, d, p.ta, q.ta, q.tb) ? std::min(m + n, int64_t{1} << 61) : std::max(m, n);
}

hipError_t launch_two(const Product &p, const Product &q, int64_t bytes, hipStream_t stream) {
    const Choice c = choice_of(p), d = choice_of(q);
    hipError_t err = hipSuccess;
    Product a = p, b = q;
    a.splits = c.splits, b.splits = d.splits;
    if (c.tile == kRows && d.tile == kRows && c.splits == 1 && d.splits == 1 &&
        launch_rows_pair(a, c.shape, b, d.shape, stream, &err))
        return err;
    const int64_t own = slices_bytes(c, p.batch, p.M, p.N);
    if (paired(c, d, p.ta, q.ta, q.tb) && own + slices_bytes(d, q.batch, q.M, q.N) <= bytes) {
        a.narrow = narrow(p), b.narrow = narrow(q);
        a.slices = c.splits > 1 ? p.space : nullptr, b.slices = d.splits > 1 ? q.space + own / 4 : nullptr;
        if (launch_tile_pair(a, b, c.tile, stream, &err)) {
            if (err != hipSuccess || (c.splits == 1 && d.splits == 1)) return err;
            if (c.splits > 1 && d.splits > 1) return launch_sum_slices(a, b, stream);
            return launch_sum_slices(c.splits > 1 ? a : b, stream);
        }
    }
    err = launch_product(p, stream);
    return err == hipSuccess ? launch_product(q, stream) : err;
}

hipError_t launch_product(const Product &asked, hipStream_t stream) {
    Product p = asked;
    p.narrow = narrow(p);
    const Choice c = choice_of(p);
    p.splits = c.splits;
    p.slices = c.splits > 1 ? p.space : nullptr;
    p.row_a = p.row_b = nullptr;
    hipError_t err = hipSuccess;
    if (c.half && p.narrow) {
        p.blocks_a = stat_blocks(p.M, p.K, !p.ta), p.blocks_b = stat_blocks(p.N, p.K, p.tb);
        p.row_a = reinterpret_cast<const RowStat *>(p.space + (c.splits > 1 ? c.splits * p.batch * p.M * p.N : 0));
        p.row_b = p.row_a + p.blocks_a * p.batch * p.M;
        err = launch_row_stats(p, stream);
    }
    if (c.tile == kRows)
        err = launch_rows(p, c.shape, stream);
    else if (err == hipSuccess)
        err = p.ta ? (p.tb ? launch_tile_tt(p, c.tile, stream) : launch_tile_tn(p, c.tile, stream))
                   : (p.tb ? launch_tile_nt(p, c.tile, stream) : launch_tile_nn(p, c.tile, stream));
    if (err != hipSuccess || p.splits == 1) return err;
    return launch_sum_slices(p, stream);
}

}  // namespace fused
}  // namespace gemm_f32_impl
