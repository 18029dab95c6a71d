// FP32 <-> MXFP4 (include/gemm_mxfp4.h).
//
// A block's scale comes from the largest magnitude alone: with E the biased
// exponent field of amax, floor(log2 amax) - 2 + 127 = E - 2, clamped at 0
// (subnormal maxima have E = 0); E = 255 marks an infinity or a NaN.  The
// conversion instruction divides by the power of two exactly, rounds to
// nearest with ties to the even code and saturates at 6.

#include <algorithm>

#include "mxfp4.h"
#include "mxfp4_device.h"

namespace gemm_f32_impl {
namespace mx {
namespace {

// Scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t E = amax_bits >> 23;
    return E == 255u ? 255u : (E > 2u ? E - 2u : 0u);
}

__device__ __forceinline__ uint32_t magnitude(float x) {
    return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// Four codes (16 bits) of four values.
__device__ __forceinline__ uint32_t codes4(f32x4 v, uint32_t e) {
    const float s = scale_of(e);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    return e == 255u ? 0u : r & 0xffffu;
}

// Largest of the 8 lanes that hold a block.
__device__ __forceinline__ uint32_t max8(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // lane ^ 2
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));  // 7 - lane of 8
    return m;
}

constexpr int kRows = 4;  // rows in flight per lane

// Blocks along the rows.  Eight lanes hold a block, four values each, so a
// wavefront reads 1 KiB of a row at once; `lx` = log2 of the lanes along a
// row (8 to 256 of the workgroup's 256).
__global__ __launch_bounds__(256) void quantize_rows_kernel(Quantize p, int lx, int tiles_x,
                                                            int64_t tiles_y, int64_t tiles) {
    const int nb = (p.cols + kBlock - 1) / kBlock, words = (nb + 3) & ~3;
    const int tx = threadIdx.x & ((1 << lx) - 1), ty = threadIdx.x >> lx;
    const int rows_wg = (256 >> lx) * kRows;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_x;
        const int64_t quad = ((t - line * tiles_x) << lx) + tx;
        const int64_t b = line / tiles_y;
        const int64_t r0 = (line - b * tiles_y) * rows_wg + ty;
        const int64_t col = quad * 4, block = quad >> 3;
        const float *X = p.X + b * p.sx;
        f32x4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + static_cast<int64_t>(i) * (256 >> lx);
            v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (r < p.rows) {
                const float *x = X + r * p.ldx + col;
                if (col + 4 <= p.cols) {
                    v[i] = *reinterpret_cast<const float4u *>(x);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        if (col + k < p.cols) v[i][k] = x[k];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + static_cast<int64_t>(i) * (256 >> lx);
            const uint32_t m = max8(max(max(magnitude(v[i][0]), magnitude(v[i][1])),
                                        max(magnitude(v[i][2]), magnitude(v[i][3]))));
            const uint32_t e = scale_byte(m);
            const uint32_t c = codes4(v[i], e);
            if (r < p.rows && block < words) {
                if (block < nb)
                    *reinterpret_cast<uint16_t *>(p.q.codes + b * p.q.sq + r * p.q.ldq + quad * 2) =
                        static_cast<uint16_t>(c);
                if ((quad & 7) == 0)
                    p.q.scales[b * p.q.ss + r * p.q.lds + block] = static_cast<uint8_t>(e);
            }
        }
    }
}

// Blocks along the columns: a lane holds one column of 32 rows, so nothing
// is exchanged between lanes and a wavefront reads 256 bytes of every row.
__global__ __launch_bounds__(256) void quantize_cols_kernel(Quantize p, int64_t tiles_x,
                                                            int64_t tiles_y, int64_t tiles) {
    const int nb = (p.rows + kBlock - 1) / kBlock, words = (nb + 3) & ~3;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_x, b = line / tiles_y;
        const int64_t block = line - b * tiles_y;
        const int64_t c = (t - line * tiles_x) * 256 + threadIdx.x;
        if (c >= p.cols) continue;
        const float *X = p.X + b * p.sx + c;
        float v[kBlock];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            const int64_t r = block * kBlock + k;
            v[k] = r < p.rows ? X[r * p.ldx] : 0.0f;
            m = max(m, magnitude(v[k]));
        }
        const uint32_t e = scale_byte(m);
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f32x4 lo{v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]};
            const f32x4 hi{v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]};
            o[k] = codes4(lo, e) | codes4(hi, e) << 16;
        }
        *reinterpret_cast<u32x4 *>(p.qt.codes + b * p.qt.sq + c * p.qt.ldq + block * kBlockBytes) = o;
        uint8_t *s = p.qt.scales + b * p.qt.ss + c * p.qt.lds;
        s[block] = static_cast<uint8_t>(e);
        if (block == nb - 1)
            for (int64_t k = nb; k < words; ++k) s[k] = 0;
    }
}

// Four values per lane: 2 bytes of codes in, 16 bytes out.
__global__ __launch_bounds__(256) void dequantize_kernel(Dequantize p, int lx, int tiles_x,
                                                         int64_t tiles_y, int64_t tiles) {
    const int tx = threadIdx.x & ((1 << lx) - 1), ty = threadIdx.x >> lx;
    const int rows_wg = (256 >> lx) * kRows;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_x;
        const int64_t quad = ((t - line * tiles_x) << lx) + tx;
        const int64_t b = line / tiles_y;
        const int64_t r0 = (line - b * tiles_y) * rows_wg + ty;
        const int64_t col = quad * 4;
        if (col >= p.cols) continue;
        uint32_t c[kRows], e[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + static_cast<int64_t>(i) * (256 >> lx);
            c[i] = e[i] = 0;
            if (r < p.rows) {
                c[i] = *reinterpret_cast<const uint16_t *>(p.q.codes + b * p.q.sq + r * p.q.ldq + quad * 2);
                e[i] = p.q.scales[b * p.q.ss + r * p.q.lds + (quad >> 3)];
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + static_cast<int64_t>(i) * (256 >> lx);
            if (r >= p.rows) continue;
            const float s = scale_of(e[i]);
            const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 0);
            const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], s, 1);
            float *y = p.Y + b * p.sy + r * p.ldy + col;
            const f32x4 v{lo[0], lo[1], hi[0], hi[1]};
            if (col + 4 <= p.cols) {
                *reinterpret_cast<float4u *>(y) = v;
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (col + k < p.cols) y[k] = v[k];
            }
        }
    }
}

// Lanes along a row: enough for the row's quads, 8 to 256.
struct Lanes {
    int lx, tiles_x;
    int64_t tiles_y, tiles;
    unsigned grid;
};
Lanes lanes_for(int64_t quads, int64_t rows, int64_t batch) {
    Lanes l{};
    l.lx = 3;
    while (l.lx < 8 && (int64_t{1} << l.lx) < quads) ++l.lx;
    l.tiles_x = static_cast<int>((quads + (int64_t{1} << l.lx) - 1) >> l.lx);
    const int64_t rows_wg = (256 >> l.lx) * kRows;
    l.tiles_y = (rows + rows_wg - 1) / rows_wg;
    l.tiles = l.tiles_x * l.tiles_y * batch;
    l.grid = static_cast<unsigned>(std::min<int64_t>(l.tiles, 1 << 22));
    return l;
}

}  // namespace

hipError_t launch_quantize(const Quantize &q, hipStream_t stream) {
    if (q.along_rows) {
        const int64_t words = (blocks_of(q.cols) + 3) / 4 * 4;
        const Lanes l = lanes_for(words * 8, q.rows, q.batch);
        quantize_rows_kernel<<<l.grid, 256, 0, stream>>>(q, l.lx, l.tiles_x, l.tiles_y, l.tiles);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (q.along_cols) {
        const int64_t tx = (q.cols + int64_t{255}) / 256, ty = blocks_of(q.rows);
        const int64_t tiles = tx * ty * q.batch;
        quantize_cols_kernel<<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 22)), 256, 0,
                               stream>>>(q, tx, ty, tiles);
        return hipGetLastError();
    }
    return hipSuccess;
}

hipError_t launch_dequantize(const Dequantize &d, hipStream_t stream) {
    const Lanes l = lanes_for((d.cols + int64_t{3}) / 4, d.rows, d.batch);
    dequantize_kernel<<<l.grid, 256, 0, stream>>>(d, l.lx, l.tiles_x, l.tiles_y, l.tiles);
    return hipGetLastError();
}

}  // namespace mx
}  // namespace gemm_f32_impl
