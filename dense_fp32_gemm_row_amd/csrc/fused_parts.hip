// What stands beside the fused tile kernels: the sum of slices, the slope of
// a layer's activation with its bias gradient, and the rest of the cross
// entropy.  All of it reads and writes its matrices once, by memory's rate.

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {
namespace {

// C = epilogue(sum of slices), an element a thread, slices in order.
__global__ __launch_bounds__(256) void sum_slices_kernel(Product p, int64_t elements) {
    const int64_t per = static_cast<int64_t>(p.M) * p.N;
    for (int64_t o = blockIdx.x * int64_t{256} + threadIdx.x; o < elements; o += gridDim.x * int64_t{256}) {
        const int64_t b = o / per, q = o - b * per, m = q / p.N, n = q - m * p.N;
        const float *W = p.slices + b * p.splits * per + q;
        float z = W[0];
        for (int s = 1; s < p.splits; ++s) z += W[s * per];
        if (p.e.bias.p != nullptr) z += p.e.bias.p[b * p.e.bias.stride + n];
        if (p.e.pre.p != nullptr) p.e.pre.p[b * p.e.pre.stride + m * p.e.pre.ld + n] = z;
        float v = activate(p.e.activation, z);
        if (p.e.residual.p != nullptr) v += p.e.residual.p[b * p.e.residual.stride + m * p.e.residual.ld + n];
        p.c.p[b * p.c.stride + m * p.c.ld + n] = v;
    }
}

// A block of rows of 256 columns: dZ, and the columns' sums over the block.
__global__ __launch_bounds__(256) void slope_kernel(Slope s, int64_t strips, int64_t units) {
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t strip = u % strips, rest = u / strips, block = rest % s.blocks, b = rest / s.blocks;
        const int64_t n = strip * 256 + threadIdx.x;
        if (n >= s.N) continue;
        const int64_t first = block * s.rows, last = min(first + s.rows, int64_t{s.M});
        float sum = 0.0f;
        for (int64_t m = first; m < last; ++m) {
            float v = s.dc.p[b * s.dc.stride + m * s.dc.ld + n];
            if (s.activation != GEMM_F32_ACT_NONE)
                v *= slope(s.activation, s.pre.p[b * s.pre.stride + m * s.pre.ld + n]);
            if (s.dz.p != nullptr) s.dz.p[b * s.dz.stride + m * s.dz.ld + n] = v;
            sum += v;
        }
        if (s.partial != nullptr) s.partial[(b * s.blocks + block) * s.N + n] = sum;
    }
}

__global__ __launch_bounds__(256) void bias_kernel(Slope s, int64_t strips, int64_t units) {
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t b = u / strips, n = (u - b * strips) * 256 + threadIdx.x;
        if (n >= s.N) continue;
        float sum = 0.0f;
        for (int q = 0; q < s.blocks; ++q) sum += s.partial[(b * s.blocks + q) * s.N + n];
        s.dbias.p[b * s.dbias.stride + n] = sum;
    }
}

// A wavefront a row: its pieces' statistics joined.
__global__ __launch_bounds__(256) void loss_kernel(Loss l) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = blockIdx.x * int64_t{4} + (threadIdx.x >> 6); t < l.T; t += gridDim.x * int64_t{4}) {
        float m = -__builtin_inff(), s = 0.0f;
        for (int g = lane; g < l.groups; g += 64) {
            const stat2 q = l.stats[t * l.groups + g];
            merge_stats(m, s, q.x, q.y);
        }
        for (int d = 1; d < 64; d *= 2) {
            const float m2 = __shfl_xor(m, d), s2 = __shfl_xor(s, d);
            merge_stats(m, s, m2, s2);
        }
        if (lane == 0) {
            const float lse = m + logf(s);
            l.lse[t] = lse;
            if (l.loss != nullptr) {
                const int64_t target = l.target[t];
                l.loss[t] = target == l.ignore ? 0.0f
                            : target >= 0 && target < l.V ? lse - l.at_target[t] : __builtin_nanf("");
            }
        }
    }
}

__global__ __launch_bounds__(256) void probabilities_kernel(Loss l, int64_t strips, int64_t units) {
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t t = u / strips, v = (u - t * strips) * 256 + threadIdx.x;
        if (v >= l.V) continue;
        const int64_t target = l.target[t];
        float p = 0.0f;
        if (target != l.ignore) {
            const float g = l.grad_loss != nullptr ? l.grad_loss[t] : 1.0f;
            p = g * (expf(l.logits[t * l.V + v] - l.lse[t]) - (v == target ? 1.0f : 0.0f));
            if (target < 0 || target >= l.V) p = __builtin_nanf("");
        }
        l.logits[t * l.V + v] = p;
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
// rows' (a row a thread).
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
            int64_t k = k0 + 4 * lane;
            for (; k + 3 < k1; k += 256) {
                const f32x4 v = *reinterpret_cast<const float4u *>(p + k);
#pragma unroll
                for (int e = 0; e < 4; ++e) count(s, v[e]);
            }
            for (; k < k1; ++k) count(s, p[k]);  // the last three at most, of one lane
            for (int d = 1; d < 64; d *= 2) join(s, __shfl_xor(s.top, d), __shfl_xor(s.count, d), __shfl_xor(s.sum, d));
            if (lane != 0) continue;
        } else {
            row = strip * 256 + tid;
            if (row >= j.rows) continue;
            p += row;
#pragma unroll 8
            for (int64_t k = k0; k < k1; ++k) count(s, p[k * j.x.ld]);
        }
        j.out[(block * batch + n) * j.rows + row] = s;
    }
}

unsigned blocks_for(int64_t n) { return static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(n, 1), 1 << 21)); }

}  // namespace

hipError_t launch_sum_slices(const Product &p, hipStream_t stream) {
    const int64_t n = p.batch * p.M * p.N;
    sum_slices_kernel<<<blocks_for(div_up(n, 256)), 256, 0, stream>>>(p, n);
    return hipGetLastError();
}

hipError_t launch_slope(const Slope &s, hipStream_t stream) {
    const int64_t strips = div_up(s.N, 256), units = strips * s.blocks * s.batch;
    slope_kernel<<<blocks_for(units), 256, 0, stream>>>(s, strips, units);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && s.dbias.p != nullptr) {
        bias_kernel<<<blocks_for(strips * s.batch), 256, 0, stream>>>(s, strips, strips * s.batch);
        err = hipGetLastError();
    }
    return err;
}

hipError_t launch_loss(const Loss &l, hipStream_t stream) {
    loss_kernel<<<blocks_for(div_up(l.T, 4)), 256, 0, stream>>>(l);
    return hipGetLastError();
}

hipError_t launch_probabilities(const Loss &l, hipStream_t stream) {
    const int64_t strips = div_up(l.V, 256), units = strips * l.T;
    probabilities_kernel<<<blocks_for(units), 256, 0, stream>>>(l, strips, units);
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

int64_t product_space(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, bool statistics) {
    const Choice c = choose(tb, batch, M, N, K, true, statistics ? kStatistics : kPlain);
    const __int128 slices = c.splits > 1 ? static_cast<__int128>(4 * c.splits) * batch * M * N : 0;
    // either form of either operand
    const __int128 stats = c.half ? static_cast<__int128>(sizeof(RowStat)) * batch *
                                        (std::max(stat_blocks(M, K, true), stat_blocks(M, K, false)) * M +
                                         std::max(stat_blocks(N, K, true), stat_blocks(N, K, false)) * N)
                                  : 0;
    return static_cast<int64_t>(std::min<__int128>(slices + stats, __int128{1} << 61));
}

hipError_t launch_product(const Product &asked, hipStream_t stream) {
    Product p = asked;
    p.narrow = narrow_operand(p.a.ld, !p.ta) && narrow_operand(p.b.ld, p.tb);
    const Choice c = choose(p.tb, p.batch, p.M, p.N, p.K, p.space != nullptr, p.mode == kStore ? kPlain : kStatistics);
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
