// C = A B^T with both operands in MXFP4 (include/gemm_mxfp4.h).

#include <algorithm>

#include "mxfp4.h"
#include "mxfp4_device.h"

namespace gemm_f32_impl {
namespace mx {
namespace {

// One wavefront per 32 x 32 tile, operands straight from global memory.  In
// v_mfma_scale_f32_32x32x64_f8f6f4 lane l holds the codes of row l % 32,
// block l / 32 of two, and the block's scale byte.
__global__ __launch_bounds__(256) void product_kernel(Product p, int64_t tiles_m, int64_t tiles_n,
                                                      int64_t tiles) {
    const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
    const int nb = (p.K + kBlock - 1) / kBlock;
    for (int64_t t = blockIdx.x * int64_t{4} + (threadIdx.x >> 6); t < tiles;
         t += gridDim.x * int64_t{4}) {
        const int64_t line = t / tiles_n, b = line / tiles_m;
        const int64_t n0 = (t - line * tiles_n) * 32, m0 = (line - b * tiles_m) * 32;
        const int64_t m = min(m0 + row, int64_t{p.M} - 1), n = min(n0 + row, int64_t{p.N} - 1);
        const uint8_t *A = p.a.codes + b * p.a.sq + m * p.a.ldq;
        const uint8_t *B = p.b.codes + b * p.b.sq + n * p.b.ldq;
        const uint8_t *As = p.a.scales + b * p.a.ss + m * p.a.lds;
        const uint8_t *Bs = p.b.scales + b * p.b.ss + n * p.b.lds;
        f32x16 acc = {};
        for (int64_t k = half; k < nb + half; k += 2) {
            u32x4 x = {}, y = {};
            int ex = 0, ey = 0;
            if (k < nb) {
                x = *reinterpret_cast<const u32x4 *>(A + k * kBlockBytes);
                y = *reinterpret_cast<const u32x4 *>(B + k * kBlockBytes);
                ex = As[k];
                ey = Bs[k];
            }
            const i32x8 X = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
            const i32x8 Y = {(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(X, Y, acc, 4, 4, 0, ex, 0, ey);
        }
        if (n0 + row < p.N) {
            float *C = p.C + b * p.sc + n0 + row;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t r = m0 + (i & 3) + 8 * (i >> 2) + 4 * half;
                if (r < p.M) C[r * p.ldc] = acc[i];
            }
        }
    }
}

}  // namespace

int product_splits(int64_t, int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_product(const Product &p, hipStream_t stream) {
    const int64_t tm = (p.M + int64_t{31}) / 32, tn = (p.N + int64_t{31}) / 32;
    const int64_t tiles = tm * tn * p.batch;
    product_kernel<<<static_cast<unsigned>(std::min<int64_t>((tiles + 3) / 4, 1 << 22)), 256, 0,
                     stream>>>(p, tm, tn, tiles);
    return hipGetLastError();
}

}  // namespace mx
}  // namespace gemm_f32_impl
