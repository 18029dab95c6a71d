// C = A op(W) with A in FP32 and W in MXFP4 (include/gemm_mxfp4.h).
//
// An FP32 significand has 24 bits and a bf16 one 8, so a value splits into
// three bf16 parts by truncation with nothing left over: a = a0 + a1 + a2.
// An element of W times its power of two is a bf16 value exactly.  Three
// bf16 products into one FP32 accumulator therefore sum the exact products
// a * w, as the FP32 matrix instructions would, at a third of the bf16 rate
// where those run at a sixteenth.

#include <algorithm>
#include <type_traits>

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

// W as stored, few rows of A, and operands of any stride: a workgroup of 8
// wavefronts holds a tile of 16 x 128, its wavefronts take steps of 32 k in
// turn, straight from global memory, and their sums are added in LDS in a
// fixed order.  In v_mfma_f32_16x16x32_bf16 lane l holds 8 k, from 8 (l / 16),
// of row (column) l % 16; here lane l reads those k of 8 neighbouring columns
// from 8 (l % 16), a word of codes for each, and turns pairs of values of two
// columns, as W holds them, into pairs of two k.  Neighbouring tiles run on
// one XCD, whose L2 then fetches lines of W, and of its scales, that tiles
// share once (16 x 4096 x 14336: 16.9 us, 18.5 without).  14336 columns x 4096
// take 16.0 us for a row and 17.7 for 16, W alone, at a copy's rate, 6.6: vector
// instructions (splitting 16 rows whatever M is, decoding, pairing columns) are
// busy 65% of the time, and with two wavefronts a SIMD what is left waits for
// loads, eight words and eight single bytes of scales a step.
constexpr int kStoredWaves = 8;
__global__ __launch_bounds__(64 * kStoredWaves) void weight_stored_kernel(Product p, int64_t tiles_m,
                                                                          int64_t tiles_n, int64_t tiles,
                                                                          int len) {
    constexpr int C = 8, NW = kStoredWaves;  // 8 columns: a word of codes
    __shared__ __align__(16) float sums[NW][C][4][64];
    const int lane = threadIdx.x & 63, row = lane & 15, group = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int steps = (p.K + kBlock - 1) / kBlock;
    for (int64_t t = xcd_remap(blockIdx.x, gridDim.x); t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_n, slice = line / tiles_m, b = slice / p.splits;
        const int64_t n0 = (t - line * tiles_n) * 16 * C, m0 = (line - slice * tiles_m) * 16;
        const int first = static_cast<int>(slice - b * p.splits) * len, last = min(first + len, steps);
        // rows and columns past the end repeat the last ones' and are not stored
        const float *A = p.x + b * p.sx + min(m0 + row, int64_t{p.M} - 1) * p.ldx;
        const int64_t n = min(n0 + C * row, int64_t{p.N - 1} / C * C);
        const uint8_t *W = p.b.codes + b * p.b.sq + n / 2;
        const uint8_t *S = p.b.scales + b * p.b.ss + n / kBlock;
        struct Step {
            float a[8];
            uint32_t w[8], e[8];
        };
        auto load = [&](int s) {
            Step v;
            const int64_t k = s * int64_t{kBlock} + 8 * group;
            const bool whole = (s + int64_t{1}) * kBlock <= p.K;
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // A past K is zero, so what W holds there does not matter
                const int64_t q = whole ? k + i : min(k + i, int64_t{p.K} - 1);
                v.w[i] = *reinterpret_cast<const uint32_t *>(W + q * p.b.ldq);
                v.e[i] = S[q * p.b.lds];
            }
            if (whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f32x4 x = *reinterpret_cast<const float4u *>(A + k + 4 * i);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v.a[4 * i + q] = x[q];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v.a[i] = k + i < p.K ? A[k + i] : 0.0f;
            }
            return v;
        };
        f32x4 acc[C];
#pragma unroll
        for (int j = 0; j < C; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        int s = first + wave;
        if (s < last) {
            Step now = load(s);
            for (; s < last; s += NW) {
                const Step next = load(min(s + NW, last - 1));
                uint32_t h[3][8];
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    split3(now.a[i], h[0][i], h[1][i], h[2][i]);
                    f[i] = scale_of(now.e[i]);
                }
                u32x4 x[3];
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    x[c] = u32x4{pack_high(h[c][0], h[c][1]), pack_high(h[c][2], h[c][3]),
                                 pack_high(h[c][4], h[c][5]), pack_high(h[c][6], h[c][7])};
                auto pair = [&](auto jc) {  // columns 2 j and 2 j + 1
                    constexpr int j = decltype(jc)::value;
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                                                now.w[i], f[i], j));
                    const u32x4 even = {(v[0] & 0xffffu) | (v[1] << 16), (v[2] & 0xffffu) | (v[3] << 16),
                                        (v[4] & 0xffffu) | (v[5] << 16), (v[6] & 0xffffu) | (v[7] << 16)};
                    const u32x4 odd = {pack_high(v[0], v[1]), pack_high(v[2], v[3]),
                                       pack_high(v[4], v[5]), pack_high(v[6], v[7])};
#pragma unroll
                    for (int q = 2; q >= 0; --q) {
                        acc[2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, x[q]), __builtin_bit_cast(bf16x8, even), acc[2 * j], 0, 0, 0);
                        acc[2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, x[q]), __builtin_bit_cast(bf16x8, odd), acc[2 * j + 1], 0, 0, 0);
                    }
                };
                pair(std::integral_constant<int, 0>{}), pair(std::integral_constant<int, 1>{});
                pair(std::integral_constant<int, 2>{}), pair(std::integral_constant<int, 3>{});
                now = next;
            }
        }
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[wave][j][r][lane] = acc[j][r];
        __syncthreads();
        float *out = p.splits > 1 ? p.W + slice * p.M * p.N : p.C + b * p.sc;
        const int64_t ldc = p.splits > 1 ? p.N : p.ldc;
        for (int o = threadIdx.x; o < C * 256; o += 64 * NW) {
            const int c = o % (16 * C), r = o / (16 * C), l = c / C + 16 * (r >> 2);
            if (m0 + r >= p.M || n0 + c >= p.N) continue;
            float v = sums[0][c % C][r & 3][l];
#pragma unroll
            for (int q = 1; q < NW; ++q) v += sums[q][c % C][r & 3][l];
            out[(m0 + r) * ldc + n0 + c] = v;
        }
        __syncthreads();
    }
}

// W transposed, few rows of A, and operands of any stride: a workgroup of 8
// wavefronts holds a tile of 16 x 16 NT, its wavefronts take steps of 128 k
// in turn, straight from global memory, and their sums are added in LDS in a
// fixed order.  In v_mfma_f32_16x16x32_bf16 lane l holds 8 k of row (column)
// l % 16; here lane group l / 16 takes block l / 16 of a step, 8 of its k in
// each of 4 instructions, so a lane's codes are 16 bytes in a row of W and
// its part of A 128 bytes.  Reading A, repeated for every 16 NT columns, bounds
// it: a lane's 16 bytes at a time lie in lines of their own, and L1 serves about
// one line a cycle (7.4 million lines at 16 rows x 14336 x 4096, 76% of all
// cycles, half of them A's; vector instructions are busy 33%).  4 rows x 14336 x
// 4096 take 15.2 us, 16 rows 18.8 (W alone, at a copy's rate, 6.6).
constexpr int kRowsWaves = 8;
template <int NT>
__global__ __launch_bounds__(64 * kRowsWaves) void weight_rows_kernel(Product p, int64_t tiles_m,
                                                                      int64_t tiles_n, int64_t tiles, int len) {
    __shared__ __align__(16) float sums[kRowsWaves][NT][4][64];
    const int lane = threadIdx.x & 63, row = lane & 15, group = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int nb = (p.K + kBlock - 1) / kBlock;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_n, slice = line / tiles_m, b = slice / p.splits;
        const int64_t n0 = (t - line * tiles_n) * 16 * NT, m0 = (line - slice * tiles_m) * 16;
        const int first = static_cast<int>(slice - b * p.splits) * len, last = min(first + len, (nb + 3) / 4);
        const float *A = p.x + b * p.sx + min(m0 + row, int64_t{p.M} - 1) * p.ldx;
        const uint8_t *W[NT], *S[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t n = min(n0 + 16 * j + row, int64_t{p.N} - 1);
            W[j] = p.b.codes + b * p.b.sq + n * p.b.ldq;
            S[j] = p.b.scales + b * p.b.ss + n * p.b.lds;
        }
        f32x4 acc[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = first + wave; s < last; s += kRowsWaves) {
            const int block = s * 4 + group;
            const int64_t held = min(block, nb - 1);
            u32x4 w[NT];
            float e[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                w[j] = *reinterpret_cast<const u32x4 *>(W[j] + held * kBlockBytes);
                e[j] = scale_of(S[j][held]);
            }
            f32x4 a[8];
            const int64_t k = block * int64_t{kBlock};
            if (s * 4 * kBlock + 4 * kBlock <= p.K) {
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const float4u *>(A + k + 4 * i);
            } else {  // A past K is zero, so what W holds there does not matter
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i / 4][i % 4] = k + i < p.K ? A[k + i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[3][8];
#pragma unroll
                for (int q = 0; q < 8; ++q) split3(a[2 * i + q / 4][q % 4], h[0][q], h[1][q], h[2][q]);
                u32x4 x[3];
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    x[c] = u32x4{pack_high(h[c][0], h[c][1]), pack_high(h[c][2], h[c][3]),
                                 pack_high(h[c][4], h[c][5]), pack_high(h[c][6], h[c][7])};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t c = w[j][i];
                    const u32x4 v = {
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e[j], 0)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e[j], 1)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e[j], 2)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e[j], 3))};
#pragma unroll
                    for (int q = 2; q >= 0; --q)
                        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, x[q]), __builtin_bit_cast(bf16x8, v), acc[j], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[wave][j][r][lane] = acc[j][r];
        __syncthreads();
        float *out = p.splits > 1 ? p.W + slice * p.M * p.N : p.C + b * p.sc;
        const int64_t ldc = p.splits > 1 ? p.N : p.ldc;
        for (int o = threadIdx.x; o < NT * 256; o += 64 * kRowsWaves) {
            const int l = o & 63, r = (o >> 6) & 3, j = o >> 8;
            const int64_t n = n0 + 16 * j + (l & 15), m = m0 + 4 * (l >> 4) + r;
            if (m >= p.M || n >= p.N) continue;
            float v = sums[0][j][r][l];
#pragma unroll
            for (int q = 1; q < kRowsWaves; ++q) v += sums[q][j][r][l];
            out[m * ldc + n] = v;
        }
        __syncthreads();
    }
}

// W transposed, MR (1 or 2) rows of A: FP32 multiply-adds.  A wavefront
// reads R rows of W, 64 blocks of each (1 KiB) at once, a block per lane; a
// lane's 32 values of A serve all of them, from LDS, where value quad i of
// lane l sits at i ^ (l / 2 % 8) so that 16 lanes touch every bank once.  The
// 64 partial sums of a row are added at the end, in an order that depends on
// sizes only.  A block costs 16 conversions and 32 MR multiply-adds.  A row x
// 14336 x 4096 takes 8.8 us, W read at 3.5 TB/s: a launch's latency and two
// chunks of K whose loads are waited for in turn.
constexpr int kVectorWaves = 4;
constexpr int kVectorRows = 2;
template <int MR>
__global__ __launch_bounds__(64 * kVectorWaves) void weight_vector_kernel(Product p, int64_t tiles_n,
                                                                          int64_t tiles) {
    constexpr int R = kVectorRows;
    constexpr int kChunk = 64 * kBlock, kThreads = 64 * kVectorWaves;
    __shared__ __align__(16) float xs[MR][kChunk];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int nb = (p.K + kBlock - 1) / kBlock;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t b = t / tiles_n;
        const int64_t n0 = ((t - b * tiles_n) * kVectorWaves + wave) * R;
        const float *A = p.x + b * p.sx;
        const uint8_t *W[R], *S[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min(n0 + r, int64_t{p.N} - 1);
            W[r] = p.b.codes + b * p.b.sq + n * p.b.ldq;
            S[r] = p.b.scales + b * p.b.ss + n * p.b.lds;
        }
        float acc[MR][R];
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[m][r] = 0.0f;
        for (int64_t k0 = 0; k0 < p.K; k0 += kChunk) {
            const int64_t block = k0 / kBlock + lane;
            const bool in = block < nb;
            u32x4 w[R];
            uint32_t e[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                w[r] = u32x4{0, 0, 0, 0};
                e[r] = 0;
                if (in) {
                    w[r] = *reinterpret_cast<const u32x4 *>(W[r] + block * kBlockBytes);
                    e[r] = S[r][block];
                }
            }
            __syncthreads();  // the last chunk has been used
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const float *a = A + min(m, p.M - 1) * p.ldx + k0;
                for (int i = threadIdx.x; i < kChunk / 4; i += kThreads) {
                    f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
                    if (k0 + 4 * i + 4 <= p.K) {
                        v = *reinterpret_cast<const float4u *>(a + 4 * i);
                    } else {
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            if (k0 + 4 * i + q < p.K) v[q] = a[4 * i + q];
                    }
                    const int l = i >> 3;
                    *reinterpret_cast<f32x4 *>(&xs[m][l * 32 + ((i & 7) ^ ((l >> 1) & 7)) * 4]) = v;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 8 values: a word of codes
                f32x4 v[MR][2];
#pragma unroll
                for (int m = 0; m < MR; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        v[m][h] = *reinterpret_cast<const f32x4 *>(
                            &xs[m][lane * 32 + ((2 * i + h) ^ ((lane >> 1) & 7)) * 4]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float s = scale_of(e[r]);
                    const f32x2 c0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r][i], s, 0);
                    const f32x2 c1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r][i], s, 1);
                    const f32x2 c2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r][i], s, 2);
                    const f32x2 c3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r][i], s, 3);
#pragma unroll
                    for (int m = 0; m < MR; ++m) {
                        float u = acc[m][r];
                        u = fmaf(v[m][0][0], c0[0], u), u = fmaf(v[m][0][1], c0[1], u);
                        u = fmaf(v[m][0][2], c1[0], u), u = fmaf(v[m][0][3], c1[1], u);
                        u = fmaf(v[m][1][0], c2[0], u), u = fmaf(v[m][1][1], c2[1], u);
                        u = fmaf(v[m][1][2], c3[0], u), u = fmaf(v[m][1][3], c3[1], u);
                        acc[m][r] = u;
                    }
                }
            }
        }
        // Each step halves the rows a lane holds: it hands one half to its
        // partner and adds the other's.
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            int bit = 32;
#pragma unroll
            for (int left = R; left > 1; left /= 2, bit /= 2)
#pragma unroll
                for (int r = 0; r < left / 2; ++r) {
                    const bool upper = lane & bit;
                    const float keep = upper ? acc[m][r + left / 2] : acc[m][r];
                    const float give = upper ? acc[m][r] : acc[m][r + left / 2];
                    acc[m][r] = keep + __shfl_xor(give, bit);
                }
            float v = acc[m][0];
#pragma unroll
            for (int d = bit; d > 0; d /= 2) v += __shfl_xor(v, d);
            // bit 5 of the lane chose between row halves, bit 4 between
            // quarters, ...: lane / (64 / R) is the row
            const int64_t n = n0 + lane / (64 / R);
            if (lane % (64 / R) == 0 && n < p.N && m < p.M) p.C[b * p.sc + m * p.ldc + n] = v;
        }
    }
}

// A tile of 2 x 2 wavefronts, each FM x FN blocks of 32 x 32, K in stages of
// 32.
//
// LDS holds a stage as bf16: the three parts of A's rows and W's columns, 32
// k (64 bytes: 4 slots of 8 k) a row.  Slot s of row r sits at s ^ (r / 4 % 4):
// 16 lanes that read one slot of 16 rows touch every bank once.  Column n of
// W is row n / FN + 64 (n % FN), so that a lane's results of one row of C are
// FN neighbours and are stored at once.
//
// A stage runs in 6 phases, a part of A times 16 k each, the smallest parts
// first.  Under a phase's products the next phase's operands are read from
// LDS, and in the first ones the next stage's values, loaded into registers D
// stages ago, are split (or decoded), written to the other buffer and their
// registers loaded again.  The one barrier lies before the last phase, under
// which the next stage's first operands are read.
//
// 4096 x 4096 x 14336, W as stored, takes 1056 us, 1144 on a slower card: 456
// and 420 TFLOP/s, that is 1.37 and 1.26 PFLOP/s of bf16 products, where a loop
// of nothing but them reaches 1.76 on random values.  Splitting and decoding share the issue slots with them: of
// a lone 64 x 128 tile's 0.48 us a stage, 0.27 are theirs.
template <int FM, int FN, bool BT, bool QUADS, int PER_CU>
__global__ __launch_bounds__(256, PER_CU) void weight_tile_kernel(Product p, int tiles_m, int tiles_n,
                                                               int chunks, int len) {
    constexpr int BM = 64 * FM, BN = 64 * FN, kRow = 64;
    constexpr int D = FM * FN <= 4 ? 2 : 1;   // stages that loads run ahead: the small tiles' are short
    constexpr int kUnits = BM / 32;           // 4 values of A per lane each
    constexpr int kWords = BN / 64;           // of codes per lane
    __shared__ __align__(1024) uint8_t a0[3 * BM * kRow];
    __shared__ __align__(1024) uint8_t a1[3 * BM * kRow];
    __shared__ __align__(1024) uint8_t w0[BN * kRow];
    __shared__ __align__(1024) uint8_t w1[BN * kRow];

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, row = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
    const Place at = place_of<BM, BN>(p, xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, chunks, len);
    const int64_t b = at.slice / p.splits;
    const int nb = (p.K + kBlock - 1) / kBlock, nbn = (p.N + kBlock - 1) / kBlock;

    const int s1 = min(at.g1 * 4, nb);  // stages are counted from K's start, 4 a chunk

    // ---- A: 8 lanes along a row, 32 rows a unit ----
    const __amdgpu_buffer_rsrc_t ar =
        buffer_of(p.x + b * p.sx + at.m0 * p.ldx, ((p.M - 1 - at.m0) * p.ldx + p.K) * 4);
    const int lda = static_cast<int>(p.ldx) * 4;
    const int ak = (tid & 7) * 4, arow = tid >> 3;
    f32x4 av[D][kUnits];
    auto load_a = [&](int u, int s, int set) {
        const int k = s * 32 + ak, at_row = (arow + 32 * u) * lda;
        if constexpr (QUADS) {
            const int off = s < s1 && k < p.K ? k * 4 : kOutside;
            av[set][u] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ar, at_row + off, 0, 0));
        } else {  // four values may end a row, and the operand
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int off = s < s1 && k + e < p.K ? (k + e) * 4 : kOutside;
                av[set][u][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(ar, at_row + off, 0, 0));
            }
        }
    };
    // k 4 q .. 4 q + 3 of a row: half a slot
    const int aslot = (((tid & 7) >> 1) ^ ((arow >> 2) & 3)) * 16 + (tid & 1) * 8;
    auto put_a = [&](int u, uint8_t *dst, int set) {
        uint32_t h[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            split3(av[set][u][e], h[0][e], h[1][e], h[2][e]);
        }
#pragma unroll
        for (int c = 0; c < 3; ++c)
            *reinterpret_cast<u32x2 *>(dst + (c * BM + arow + 32 * u) * kRow + aslot) =
                u32x2{pack_high(h[c][0], h[c][1]), pack_high(h[c][2], h[c][3])};
    };

    // ---- W ----
    // Transposed: a lane has (part of) a column's block, kWords words of codes.
    // As stored: FN columns of 8 rows k.
    const __amdgpu_buffer_rsrc_t wr =
        BT ? buffer_of(p.b.codes + b * p.b.sq + at.n0 * p.b.ldq,
                       (p.N - 1 - at.n0) * p.b.ldq + nb * kBlockBytes)
           : buffer_of(p.b.codes + b * p.b.sq, (p.K - 1) * p.b.ldq + nbn * kBlockBytes);
    const __amdgpu_buffer_rsrc_t wsr =
        BT ? buffer_of(p.b.scales + b * p.b.ss + at.n0 * p.b.lds, (p.N - 1 - at.n0) * p.b.lds + (nb + 3) / 4 * 4)
           : buffer_of(p.b.scales + b * p.b.ss, (p.K - 1) * p.b.lds + nbn);
    const int ldq = static_cast<int>(p.b.ldq), lds = static_cast<int>(p.b.lds);
    // Transposed, the codes of 4 stages (64 bytes of a column) are loaded at
    // once, and their scales as one word: a stage's 16 bytes alone would fetch
    // the same line from L2 in every stage.
    uint32_t wc[BT ? 4 * kWords : 8 * D], we[BT ? 1 : 8 * D], wc_next[BT ? 4 * kWords : 1], we_next = 0;
    constexpr int kParts = 4 / FN;  // lanes that share a column's block
    // transposed: LDS row of the lane, its column
    const int trow = tid / kParts, tcol = FN * (trow & 63) + (trow >> 6), tpart = tid % kParts;
    auto load_group = [&](int g) {  // transposed: stages 4 g .. 4 g + 3
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 4 * g + i;
            const int off = s < s1 ? s * kBlockBytes + tpart * kWords * 4 : kOutside;
            if constexpr (FN == 4) {
                const u32x4 v = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, tcol * ldq + off, 0, 0));
#pragma unroll
                for (int q = 0; q < 4; ++q) wc_next[i * 4 + q] = v[q];
            } else {
                const u32x2 v = __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_raw_buffer_load_b64(wr, tcol * ldq + off, 0, 0));
                wc_next[2 * i] = v[0], wc_next[2 * i + 1] = v[1];
            }
        }
        we_next = __builtin_amdgcn_raw_buffer_load_b32(wsr, tcol * lds + (4 * g < s1 ? 4 * g : kOutside), 0, 0);
    };
    auto take_group = [&](int g) {
#pragma unroll
        for (int q = 0; q < 4 * kWords; ++q) wc[q] = wc_next[q];
        const int valid = min(max(s1 - 4 * g, 0), 4);  // past them the word may hold anything
        we[0] = we_next & (valid == 4 ? 0xffffffffu : (1u << (8 * valid)) - 1u);
    };
    auto load_w = [&](int s, int set) {  // as stored: one stage
        const bool live = s < s1;
        const int n = at.n0 + FN * lane;  // first column of the lane
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = s * 32 + wave * 8 + i;
            const bool in = live && k < p.K;
            const int oc = in ? k * ldq + n / 2 : kOutside, os = in ? k * lds + n / kBlock : kOutside;
            wc[8 * set + i] = FN == 4 ? __builtin_amdgcn_raw_buffer_load_b16(wr, oc, 0, 0)
                            : __builtin_amdgcn_raw_buffer_load_b8(wr, oc, 0, 0);
            we[8 * set + i] = __builtin_amdgcn_raw_buffer_load_b8(wsr, os, 0, 0);
        }
    };
    auto put_w = [&](auto ic, uint8_t *dst) {  // stage ic of 4
        constexpr int of = decltype(ic)::value;
        if constexpr (BT) {
            const float e = scale_of((we[0] >> (8 * of)) & 255u);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t c = wc[of * kWords + i];
                const u32x4 v = {
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 3))};
                const int slot = (tpart * kWords + i) ^ ((trow >> 2) & 3);
                *reinterpret_cast<u32x4 *>(dst + trow * kRow + slot * 16) = v;
            }
        } else {
            uint32_t v[8][FN / 2];  // pairs of columns of row k
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = wc[of % D * 8 + i];
                const float e = scale_of(we[of % D * 8 + i]);
                v[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 0));
                if constexpr (FN == 4)
                    v[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, e, 1));
            }
#pragma unroll
            for (int c = 0; c < FN; ++c) {
                u32x4 o;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t lo = v[2 * q][c / 2], hi = v[2 * q + 1][c / 2];
                    o[q] = c & 1 ? pack_high(lo, hi) : (lo & 0xffffu) | (hi << 16);
                }
                const int r = lane + 64 * c, slot = wave ^ ((r >> 2) & 3);
                *reinterpret_cast<u32x4 *>(dst + r * kRow + slot * 16) = o;
            }
        }
    };

    // ---- products ----
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    u32x4 x[2][FM], y[2][FN];
    const int ra = (wm * FM * 32 + row) * kRow, rw = (wn * 32 + row) * kRow, sw = (row >> 2) & 3;
    auto fetch = [&](auto pc, const uint8_t *a, const uint8_t *w) {  // operands of a phase
        constexpr int ph = decltype(pc)::value, ks = ph / 3, part = 2 - ph % 3;
        const int slot = ((2 * ks + half) ^ sw) * 16;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            x[ph & 1][i] = *reinterpret_cast<const u32x4 *>(a + part * BM * kRow + ra + 32 * i * kRow + slot);
        if constexpr (ph % 3 == 0)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                y[ks][j] = *reinterpret_cast<const u32x4 *>(w + rw + 64 * j * kRow + slot);
    };
    auto multiply = [&](auto pc) {
        constexpr int ph = decltype(pc)::value, ks = ph / 3;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int k = 0; k < FN; ++k) {
                const int j = i & 1 ? FN - 1 - k : k;
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, x[ph & 1][i]), __builtin_bit_cast(bf16x8, y[ks][j]),
                    acc[i][j], 0, 0, 0);
            }
    };
    // Between two matrix instructions: an LDS read, a few vector instructions
    // of the splitting, and its writes and loads.
    auto interleave = [&]() {
#pragma unroll
        for (int k = 0; k < FM * FN; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
            __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        // The sums so far are used here, so their instructions stay ahead.
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) asm volatile("" ::"a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
    };

    constexpr std::integral_constant<int, 0> p0;
    constexpr std::integral_constant<int, 1> p1;
    constexpr std::integral_constant<int, 2> p2;
    constexpr std::integral_constant<int, 3> p3;
    constexpr std::integral_constant<int, 4> p4;
    constexpr std::integral_constant<int, 5> p5;

    // Stage s (the ic-th of its group) in (a, w); stage s + 1, in registers,
    // goes to (na, nw).
    auto stage = [&](auto ic, int s, const uint8_t *a, const uint8_t *w, uint8_t *na, uint8_t *nw) {
        constexpr int i = decltype(ic)::value;
        auto units = [&](int first, int last) {
#pragma unroll
            for (int u = first; u < last; ++u) {
                put_a(u, na, (i + 1) % D);
                load_a(u, s + 1 + D, (i + 1) % D);
            }
        };
        fetch(p1, a, w);
        units(0, kUnits / 4);
        multiply(p0);
        interleave();
        fetch(p2, a, w);
        units(kUnits / 4, kUnits / 2);
        multiply(p1);
        interleave();
        fetch(p3, a, w);
        units(kUnits / 2, 3 * kUnits / 4);
        multiply(p2);
        interleave();
        fetch(p4, a, w);
        units(3 * kUnits / 4, kUnits);
        multiply(p3);
        interleave();
        fetch(p5, a, w);
        put_w(std::integral_constant<int, (i + 1) % 4>{}, nw);
        if constexpr (!BT) {
            load_w(s + 1 + D, (i + 1) % D);
        } else if constexpr (i == 0) {
            load_group(s / 4 + 1);
        } else if constexpr (i == 2) {
            take_group(s / 4 + 1);
        }
        multiply(p4);
        interleave();
        wait_older<63>();  // LDS accesses alone
        barrier_only();
        fetch(p0, na, nw);
        multiply(p5);
        interleave();
    };

    int s = 4 * at.g0;
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) load_a(u, s + d, d);
        if constexpr (!BT) load_w(s + d, d);
    }
    if constexpr (BT) {
        load_group(s / 4);
        take_group(s / 4);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        put_a(u, a0, 0);
        load_a(u, s + D, 0);
    }
    put_w(p0, w0);
    if constexpr (!BT) load_w(s + D, 0);
    wait_older<63>();
    barrier_only();
    fetch(p0, a0, w0);
    for (; s + 3 < s1; s += 4) {
        stage(p0, s, a0, w0, a1, w1);
        stage(p1, s + 1, a1, w1, a0, w0);
        stage(p2, s + 2, a0, w0, a1, w1);
        stage(p3, s + 3, a1, w1, a0, w0);
    }
    if (s < s1) {
        stage(p0, s, a0, w0, a1, w1);
        if (s + 1 < s1) {
            stage(p1, s + 1, a1, w1, a0, w0);
            if (s + 2 < s1) stage(p2, s + 2, a0, w0, a1, w1);
        }
    }

    // ---- results: FN neighbours a lane ----
    const int64_t ldc = p.splits > 1 ? p.N : p.ldc;
    const float *base = p.splits > 1 ? p.W + at.slice * p.M * ldc : p.C + at.slice * p.sc;
    const int mw = at.m0 + wm * FM * 32, n = at.n0 + FN * (32 * wn + row);
    if (mw >= p.M || n >= p.N) return;
    const __amdgpu_buffer_rsrc_t c = buffer_of(base + mw * ldc, ((p.M - 1 - mw) * ldc + p.N) * 4);
    const int ld = static_cast<int>(ldc) * 4;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float v[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) v[j] = acc[i][j][r];
            store_neighbours<FN>(v, c, (32 * i + (r & 3) + 8 * (r >> 2) + 4 * half) * ld + n * 4, p.N - n);
        }
}

// PER_CU workgroups of a CU, for the registers that a wavefront may take.
// Where the 128 x 256 tile's do not fit two without spilling dozens (W as
// stored fits by itself), the compiler is not held to two: with K % 4 != 0
// and W as stored 4096 x 4096 x 14335 took 1387 us held to them, 1153 so; with
// W transposed and K % 4 == 0 a few spills cost less than the second
// workgroup brings (1004 us against 1052).  With W transposed and K % 4 != 0 the
// registers left to themselves are 268, one workgroup a CU (4096 x 4096 x 14335:
// 1180 us, as stored, with two, 1165).
template <int FM, int FN, int PER_CU>
hipError_t launch_tile(const Product &p, hipStream_t stream) {
    const int tm = ceil_div(p.M, 64 * FM), tn = ceil_div(p.N, 64 * FN);
    const int chunks = ceil_div(static_cast<int>(blocks_of(p.K)), 4), len = ceil_div(chunks, p.splits);
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(tm) * tn * p.batch * p.splits);
    const bool quads = p.K % 4 == 0;
    auto go = [&](auto bt, auto wh) {
        constexpr bool kFits = FM * FN < 8 || (decltype(bt)::value && decltype(wh)::value);
        weight_tile_kernel<FM, FN, decltype(bt)::value, decltype(wh)::value, kFits ? PER_CU : 1>
            <<<grid, 256, 0, stream>>>(p, tm, tn, chunks, len);
    };
    if (p.b_transposed)
        quads ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else
        quads ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

template <int NT>
hipError_t launch_rows(const Product &p, hipStream_t stream) {
    const int64_t tm = (p.M + int64_t{15}) / 16, tn = (p.N + int64_t{16 * NT - 1}) / (16 * NT);
    const int64_t tiles = tm * tn * p.batch * p.splits, steps = (blocks_of(p.K) + 3) / 4;
    weight_rows_kernel<NT><<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20)), 64 * kRowsWaves, 0,
                             stream>>>(p, tm, tn, tiles, static_cast<int>((steps + p.splits - 1) / p.splits));
    return hipGetLastError();
}

template <int MR>
hipError_t launch_vector(const Product &p, hipStream_t stream) {
    constexpr int kCols = kVectorWaves * kVectorRows;
    const int64_t tn = (p.N + int64_t{kCols - 1}) / kCols, tiles = tn * p.batch;
    weight_vector_kernel<MR><<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20)),
                               64 * kVectorWaves, 0, stream>>>(p, tn, tiles);
    return hipGetLastError();
}

hipError_t launch_stored(const Product &p, hipStream_t stream) {
    const int64_t tm = (p.M + int64_t{15}) / 16, tn = (p.N + int64_t{127}) / 128;
    const int64_t tiles = tm * tn * p.batch * p.splits;
    const int len = static_cast<int>((blocks_of(p.K) + p.splits - 1) / p.splits);
    weight_stored_kernel<<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20)), 64 * kStoredWaves, 0,
                           stream>>>(p, tm, tn, tiles, len);
    return hipGetLastError();
}

}  // namespace

int weight_splits(bool b_transposed, int64_t batch, int64_t M, int64_t N, int64_t K) {
    return weight_choice::choose(b_transposed, batch, M, N, K, kMostSplits).splits;
}

hipError_t launch_weight(const Product &asked, hipStream_t stream) {
    Product p = asked;
    using namespace weight_choice;
    Choice c = choose(p.b_transposed, p.batch, p.M, p.N, p.K, p.splits > 1 ? kMostSplits : 1);
    if (c.tile != kDirect && !tiles_fit(p.b_transposed, p.batch, p.M, p.N, p.K, p.ldx, std::max(p.b.ldq, p.b.lds),
                                        std::max(p.ldc, int64_t{p.N})))
        c = {kDirect, 1, p.b_transposed ? 4 : 8};
    p.splits = c.splits;
    hipError_t err;
    if (c.tile == kDirect && !p.b_transposed)
        err = launch_stored(p, stream);
    else if (c.tile == kDirect && p.M <= 2)
        // One and two rows of A cost the vector units less than splitting 16:
        // a row x 14336 x 4096 8.8 us, against 13.7.
        err = p.M == 1 ? launch_vector<1>(p, stream) : launch_vector<2>(p, stream);
    else if (c.tile == kDirect)
        err = c.nt == 4   ? launch_rows<4>(p, stream)
              : c.nt == 2 ? launch_rows<2>(p, stream)
                          : launch_rows<1>(p, stream);
    else
        err = c.tile == 0   ? launch_tile<2, 4, 2>(p, stream)
              : c.tile == 1 ? launch_tile<1, 4, 2>(p, stream)
                            : launch_tile<1, 2, 3>(p, stream);
    if (err == hipSuccess && p.splits > 1) err = launch_sum_slices(p, stream);
    return err;
}

}  // namespace mx
}  // namespace gemm_f32_impl
