// C = A op(W) with A in FP32 and W in MXFP4 (include/gemm_mxfp4.h).
//
// An FP32 significand has 24 bits and a bf16 one 8, so a value splits into
// three bf16 parts by truncation with nothing left over: a = a0 + a1 + a2.
// An element of W times its power of two is a bf16 value exactly.  Three
// bf16 products into one FP32 accumulator therefore sum the exact products
// a * w, as the FP32 matrix instructions would, at a third of the bf16 rate
// where those run at a sixteenth.

#include <algorithm>

#include "mxfp4.h"
#include "mxfp4_device.h"

namespace gemm_f32_impl {
namespace mx {
namespace {

// The three parts of x, as the high halves of words.  An infinity is its own
// first part (inf - inf would make the rest NaN); a NaN stays one in the rest.
__device__ __forceinline__ void split3(float x, uint32_t &h0, uint32_t &h1, uint32_t &h2) {
    h0 = __builtin_bit_cast(uint32_t, x) & 0xffff0000u;
    float r = x - __builtin_bit_cast(float, h0);
    if (__builtin_fabsf(x) == __builtin_inff()) r = 0.0f;
    h1 = __builtin_bit_cast(uint32_t, r) & 0xffff0000u;
    h2 = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, h1));
}

__device__ __forceinline__ uint32_t pack_high(uint32_t lo, uint32_t hi) {
    return (lo >> 16) | (hi & 0xffff0000u);
}

// One wavefront per 32 x 32 tile.  In v_mfma_f32_32x32x16_bf16 lane l holds
// 8 consecutive k from 8 (l / 32) of row (column) l % 32.
template <bool BT>
__global__ __launch_bounds__(256) void weight_kernel(Product p, int64_t tiles_m, int64_t tiles_n,
                                                     int64_t tiles) {
    const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
    for (int64_t t = blockIdx.x * int64_t{4} + (threadIdx.x >> 6); t < tiles;
         t += gridDim.x * int64_t{4}) {
        const int64_t line = t / tiles_n, b = line / tiles_m;
        const int64_t n0 = (t - line * tiles_n) * 32, m0 = (line - b * tiles_m) * 32;
        const int64_t m = min(m0 + row, int64_t{p.M} - 1), n = min(n0 + row, int64_t{p.N} - 1);
        const float *A = p.x + b * p.sx + m * p.ldx;
        const uint8_t *W = p.b.codes + b * p.b.sq;
        const uint8_t *S = p.b.scales + b * p.b.ss;
        f32x16 acc = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
            const int64_t k = k0 + 8 * half;
            uint32_t a[3][8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                split3(k + i < p.K ? A[k + i] : 0.0f, a[0][i], a[1][i], a[2][i]);
            u32x4 w = {};
            if (BT) {
                if (k < p.K) {
                    const uint32_t c = *reinterpret_cast<const uint32_t *>(W + n * p.b.ldq + k / 2);
                    const float s = scale_of(S[n * p.b.lds + k / kBlock]);
                    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
                    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
                    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
                    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (k + i >= p.K) continue;
                    const uint32_t c = W[(k + i) * p.b.ldq + n / 2] >> (4 * (n & 1)) & 15;
                    const float s = scale_of(S[(k + i) * p.b.lds + n / kBlock]);
                    const uint32_t v = __builtin_bit_cast(
                        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
                    w[i / 2] |= (v & 0xffffu) << (16 * (i & 1));
                }
            }
#pragma unroll
            for (int s = 2; s >= 0; --s) {
                const u32x4 x = {pack_high(a[s][0], a[s][1]), pack_high(a[s][2], a[s][3]),
                                 pack_high(a[s][4], a[s][5]), pack_high(a[s][6], a[s][7])};
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x),
                                                              __builtin_bit_cast(bf16x8, w), acc, 0,
                                                              0, 0);
            }
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

int weight_splits(bool, int64_t, int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_weight(const Product &p, hipStream_t stream) {
    const int64_t tm = (p.M + int64_t{31}) / 32, tn = (p.N + int64_t{31}) / 32;
    const int64_t tiles = tm * tn * p.batch;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((tiles + 3) / 4, 1 << 22));
    if (p.b_transposed)
        weight_kernel<true><<<grid, 256, 0, stream>>>(p, tm, tn, tiles);
    else
        weight_kernel<false><<<grid, 256, 0, stream>>>(p, tm, tn, tiles);
    return hipGetLastError();
}

}  // namespace mx
}  // namespace gemm_f32_impl
