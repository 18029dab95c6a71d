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
// row (8 to 256 of the workgroup's 256).  Memory bounds it: 8192 x 4096 in
// 23.2 us (X in and codes out at 6.6 TB/s, part of X from the last-level
// cache); a row of 4096 2.3 us, the latency of a launch and a load.
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

// Blocks along the columns, and with ROWS along the rows too, in one read: a
// workgroup takes 128 x 128 values, a wavefront 32 of the rows, a lane 16 of
// those and 4 columns.  A column's block then lies in two lanes, a row's in
// 8.  (32 rows a lane would need no exchange for a column, but held 256
// registers.)  The codes of 4 blocks of a column meet in LDS so that they leave
// as 64 bytes: 16 at a time, each to a row of its own, would be partial writes
// of memory's lines.  Lanes conflict where they write there, four to a bank:
// 960 of a CU's 42,000 cycles at 4096 x 4096.
//
// Both ways the kernel takes 194 registers, so a CU holds two workgroups, and
// waits for memory: 4096 x 4096 in 20.2 us (4.2 TB/s), against 31.8 for one
// launch along each axis; vector instructions are busy 40% of the time.  Along
// the columns alone it takes 122, four workgroups a CU: 4096 x 4096 in 14.1 us
// and 8192 x 4096 in 23.9 (6.4 TB/s, part of X from the last-level cache).
// 1000 x 777 takes 8.4 us both ways, 6.5 along the columns: a workgroup's
// chain of one load, maxima, conversions and stores.
template <bool ROWS>
__global__ __launch_bounds__(256) void quantize_cols_kernel(Quantize p, int64_t tiles_x,
                                                            int64_t tiles_y, int64_t tiles) {
    constexpr int kSide = 128, kHold = 16;
    __shared__ __align__(16) uint8_t codes[kSide * 4 * kBlockBytes];  // [column][block, swizzled]
    __shared__ __align__(4) uint8_t scales[kSide * 4];                // [column][block]
    const int nbr = (p.rows + kBlock - 1) / kBlock, nbc = (p.cols + kBlock - 1) / kBlock;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5, quad = lane & 31;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_x, b = line / tiles_y;
        const int64_t slab = line - b * tiles_y, c0 = (t - line * tiles_x) * kSide;
        const int64_t col = c0 + 4 * quad, r0 = slab * kSide + wave * 32 + half * kHold;
        const float *X = p.X + b * p.sx + col;
        f32x4 v[kHold];
        if (col + 4 <= p.cols && r0 + kHold <= p.rows) {
#pragma unroll
            for (int k = 0; k < kHold; ++k) v[k] = *reinterpret_cast<const float4u *>(X + (r0 + k) * p.ldx);
        } else {
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[k][i] = r0 + k < p.rows && col + i < p.cols ? X[(r0 + k) * p.ldx + i] : 0.0f;
            }
        }
        if (ROWS) {
            const int64_t block = col / kBlock;
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const uint32_t m = max8(max(max(magnitude(v[k][0]), magnitude(v[k][1])),
                                            max(magnitude(v[k][2]), magnitude(v[k][3]))));
                const uint32_t e = scale_byte(m), c = codes4(v[k], e);
                const int64_t r = r0 + k;
                if (r < p.rows && block < ((nbc + 3) & ~3)) {
                    if (block < nbc)
                        *reinterpret_cast<uint16_t *>(p.q.codes + b * p.q.sq + r * p.q.ldq + col / 2) =
                            static_cast<uint16_t>(c);
                    if ((lane & 7) == 0)
                        p.q.scales[b * p.q.ss + r * p.q.lds + block] = static_cast<uint8_t>(e);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < kHold; ++k) m = max(m, magnitude(v[k][i]));
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
            const uint32_t e = scale_byte(m);
            u32x2 o;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4 lo{v[8 * k][i], v[8 * k + 1][i], v[8 * k + 2][i], v[8 * k + 3][i]};
                const f32x4 hi{v[8 * k + 4][i], v[8 * k + 5][i], v[8 * k + 6][i], v[8 * k + 7][i]};
                o[k] = codes4(lo, e) | codes4(hi, e) << 16;
            }
            const int c = 4 * quad + i;
            *reinterpret_cast<u32x2 *>(&codes[(c * 4 + (wave ^ (quad & 3))) * kBlockBytes + 8 * half]) = o;
            if (half == 0) scales[c * 4 + wave] = static_cast<uint8_t>(e);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSide * 4 / 256; ++i) {
            const int at = i * 256 + threadIdx.x, c = at >> 2, part = at & 3;
            const int64_t block = slab * 4 + part;
            if (c0 + c < p.cols && block < nbr)
                *reinterpret_cast<u32x4 *>(p.qt.codes + b * p.qt.sq + (c0 + c) * p.qt.ldq + block * kBlockBytes) =
                    *reinterpret_cast<const u32x4 *>(&codes[(c * 4 + (part ^ (c >> 2 & 3))) * kBlockBytes]);
        }
        if (threadIdx.x < kSide && c0 + threadIdx.x < p.cols)
            *reinterpret_cast<uint32_t *>(p.qt.scales + b * p.qt.ss + (c0 + threadIdx.x) * p.qt.lds + slab * 4) =
                *reinterpret_cast<const uint32_t *>(&scales[threadIdx.x * 4]);
        __syncthreads();
    }
}

// Four values per lane: 2 bytes of codes in, 16 bytes out, streamed past the
// caches if rows are whole lines (8192 x 14336: 102 us with ordinary stores,
// 77 so; 8192 x 4095: 24.6 with them, 33.3 streamed).  Memory bounds it:
// 8192 x 4096 in 23.9 us (6.4 TB/s); a row of 4096 2.1 us.
template <bool LINES>
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
                if constexpr (LINES)
                    __builtin_nontemporal_store(v, reinterpret_cast<float4u *>(y));
                else
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
    const int64_t words = (blocks_of(q.cols) + 3) / 4 * 4;
    if (!q.along_cols) {
        const Lanes l = lanes_for(words * 8, q.rows, q.batch);
        quantize_rows_kernel<<<l.grid, 256, 0, stream>>>(q, l.lx, l.tiles_x, l.tiles_y, l.tiles);
        return hipGetLastError();
    }
    const int64_t tx = ((q.along_rows ? words * kBlock : q.cols) + int64_t{127}) / 128;
    const int64_t ty = (q.rows + int64_t{127}) / 128, tiles = tx * ty * q.batch;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 22));
    if (q.along_rows)
        quantize_cols_kernel<true><<<grid, 256, 0, stream>>>(q, tx, ty, tiles);
    else
        quantize_cols_kernel<false><<<grid, 256, 0, stream>>>(q, tx, ty, tiles);
    return hipGetLastError();
}

hipError_t launch_dequantize(const Dequantize &d, hipStream_t stream) {
    const Lanes l = lanes_for((d.cols + int64_t{3}) / 4, d.rows, d.batch);
    if (d.ldy % 32 == 0 && d.sy % 32 == 0 && reinterpret_cast<uintptr_t>(d.Y) % 128 == 0)
        dequantize_kernel<true><<<l.grid, 256, 0, stream>>>(d, l.lx, l.tiles_x, l.tiles_y, l.tiles);
    else
        dequantize_kernel<false><<<l.grid, 256, 0, stream>>>(d, l.lx, l.tiles_x, l.tiles_y, l.tiles);
    return hipGetLastError();
}

}  // namespace mx
}  // namespace gemm_f32_impl
