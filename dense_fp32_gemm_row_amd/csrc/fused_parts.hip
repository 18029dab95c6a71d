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

hipError_t launch_product(const Product &asked, hipStream_t stream) {
    Product p = asked;
    p.narrow = narrow_operand(p.a.ld, !p.ta) && narrow_operand(p.b.ld, p.tb);
    const Choice c = choose(p.batch, p.M, p.N, p.K, p.splits);
    p.splits = c.splits;
    const hipError_t err = p.ta ? (p.tb ? launch_tile_tt(p, c.tile, stream) : launch_tile_tn(p, c.tile, stream))
                                : (p.tb ? launch_tile_nt(p, c.tile, stream) : launch_tile_nn(p, c.tile, stream));
    if (err != hipSuccess || p.splits == 1) return err;
    return launch_sum_slices(p, stream);
}

}  // namespace fused
}  // namespace gemm_f32_impl
