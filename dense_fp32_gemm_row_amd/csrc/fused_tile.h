// The tile kernel of the fused products: C = epilogue(op(A) op(B)), or the row
// statistics of the cross entropy, for a tile of C that a workgroup holds in
// registers.  Each operand form is compiled in a source file of its own.
//
// A product of FP32 values is six of bf16 parts, or three of fp16 parts, on matrix units
// that are 16 times as quick as the FP32 ones, so 2.7 (5.3) times their rate is what the
// arithmetic leaves; the parts are made once a workgroup, on the way into LDS.
//   - 256 x 256, 8 wavefronts of 128 x 64, one workgroup a CU: the fewest values split and
//     LDS reads a product.  4096 x 4096 x 4096 with bf16 parts 586 us (235 TFLOP/s), with
//     fp16 parts 347 (396; the matrix units 72% busy at 1.73 GHz), and 26 for the rows'
//     ranges; an FP32 library product takes 915.  Power holds the clock there.  At a tile's end
//     64 of a lane's 128 sums go to scratch and back (131 KB a workgroup: one path serves the
//     test for infinities, the sums by FP32 multiplies and the results), about 30 us a tile
//     with the results' stores, which nothing overlaps.
//   - 128 x 128, 4 wavefronts, two workgroups a CU (517 x 32000 x 1024 160 us in fp16 parts,
//     212 TFLOP/s; with rows that are not whole lines, 32003 x 1001, 174), and 64 x 128, three: for fewer tiles.
//     There splitting, LDS and the products take turns in one or two wavefronts a
//     SIMD: 128 x 128 x k a CU in 36 ns a k, 64 x 128 x k in 23 (matrix units a third busy).
//     1000 x 1023 x 777 in two slices of K 24 us and 5 for their sum, 37 x 4096 x 14336 in
//     16 slices 50 (4.7 TB/s of B) and 5.
//   - Tried: FP32 matrix instructions straight from memory in tiles of 64 x 64, 8
//     wavefronts sharing K (1000 x 1023 x 777 27.6 us; behind these at all of 200 sizes but ten).
#pragma once

#include <type_traits>

#include "fused_device.h"

namespace gemm_f32_impl {
namespace fused {

// LDS holds rows (of op(A), columns of op(B)) in groups of 64 in an order of
// its own: place 32 f + 16 h + i of a group is row 4 i + 2 h + f.  A lane
// that takes places j and 32 + j of a group so holds two neighbouring columns
// of C, and its half wavefront 64 of them, which are stored as a piece; and a lane that
// stages 4 neighbouring rows writes to 4 places 16 apart, next to its
// neighbours'.
__device__ __forceinline__ int row_at(int place) {
    return (place & ~63) + 4 * (place & 15) + ((place >> 3) & 2) + ((place >> 5) & 1);
}
__device__ __forceinline__ int place_of_row(int row) {
    return (row & ~63) + ((row >> 2) & 15) + ((row & 2) << 3) + ((row & 1) << 5);
}

template <int WM, int WN, int FM>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int BM = 32 * FM * WM, BN = 64 * WN;
    static constexpr bool kHalf = FM > 1;  // the tiles with a loop for fp16 parts
};

// Elements of one k range of an operand's tile, rows and k past the end zero.
// KC: k is contiguous (A as stored, B transposed).
template <bool KC>
__device__ __forceinline__ float element(const float *p, int64_t ld, int row, int rows, int k, int k1) {
    if (row >= rows || k >= k1) return 0.0f;
    return KC ? p[row * ld + k] : p[k * ld + row];
}

// Bytes from 8 k of all rows to the next 8 k of them.  A few more than those take: 16
// lanes write 64 / STAGE rows of STAGE / 8 such planes at once, to banks of their own.
constexpr int plane(int rows, int stage) { return rows * 16 + 1024 / stage; }

// A thread's share of the stages of one operand, STAGE k each: 4 consecutive k of
// kUnits rows.  Where k is contiguous (KC) these are 16-byte loads, STAGE / 4
// lanes a row; where rows are, kUnits neighbouring rows at 4 k.  Every address
// stays inside the operand: rows past its end repeat the last ones, which then
// are written to LDS where those belong.  HALF: in two fp16 parts, not three of
// bf16.  The values of D stages are held, or on their way.
template <int ROWS, int THREADS, bool KC, int STAGE, bool HALF, int D = 1>
struct Share {
    static constexpr int E = ROWS * STAGE / THREADS;  // elements
    static constexpr int kUnits = E / 4;
    static constexpr int kPlane = plane(ROWS, STAGE);  // 8 k of every row
    static constexpr int kPart = STAGE / 8 * kPlane;
    const char *base;  // of the operand's tile at k = 0
    int64_t row;       // bytes of a row of storage
    uint32_t off[KC ? kUnits : 1];
    int lds[KC ? 1 : kUnits];  // byte in a part
    float scale[HALF ? kUnits : 1];
    float v[D][E];

    __device__ __forceinline__ Share(const float *p, int64_t ld, int rows, bool more, int tid, const int *exponents) {
        row = 4 * ld;
        if constexpr (KC) {
            base = reinterpret_cast<const char *>(p);
            const int q = tid % (STAGE / 4), place = tid / (STAGE / 4);
            lds[0] = (q >> 1) * kPlane + place * 16 + (q & 1) * 8;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int r = row_at(place + u * (THREADS * 4 / STAGE));
                off[u] = static_cast<uint32_t>(min(r, rows - 1)) * static_cast<uint32_t>(row) + 16 * q;
                if constexpr (HALF) scale[u] = power(exponents[r]);
            }
        } else {
            constexpr int kLanes = ROWS / kUnits;
            const int j = tid % kLanes, q = tid / kLanes;
            // fewer last rows than a thread loads come with some from before the tile
            const int back = rows < kUnits && more ? kUnits - rows : 0;
            const int r = min(kUnits * j, rows - kUnits + back);
            base = reinterpret_cast<const char *>(p - back);
            off[0] = static_cast<uint32_t>(4 * q) * static_cast<uint32_t>(row) + 4 * r;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int at = (r - back + u + ROWS) % ROWS;
                lds[u] = (q >> 1) * kPlane + place_of_row(at) * 16 + (q & 1) * 8;
                if constexpr (HALF) scale[u] = power(exponents[at]);
            }
        }
    }
    // 2^(141 - e): values with exponent field e and less come below 2^15
    static __device__ __forceinline__ float power(int e) { return __builtin_bit_cast(float, (268 - e) << 23); }
    // The STAGE k from k on.
    __device__ __forceinline__ void load(int k, int set = 0) {
        const char *at = base + (KC ? int64_t{4} : row) * k;
        if constexpr (KC) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const f32x4 x = *reinterpret_cast<const float4u *>(at + off[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[set][4 * u + i] = x[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char *from = at + i * row + off[0];
                if constexpr (kUnits == 4) {
                    const f32x4 x = *reinterpret_cast<const float4u *>(from);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[set][4 * u + i] = x[u];
                } else if constexpr (kUnits == 2) {
                    const f32x2 x = *reinterpret_cast<const float2u *>(from);
                    v[set][i] = x[0], v[set][4 + i] = x[1];
                } else {
                    v[set][i] = *reinterpret_cast<const float *>(from);
                }
            }
        }
    }
    // The first `drop` k are zero.
    __device__ __forceinline__ void cut(int drop, int tid, int set = 0) {
        const int q = KC ? tid % (STAGE / 4) : tid / (ROWS / kUnits);
#pragma unroll
        for (int e = 0; e < E; ++e) v[set][e] = 4 * q + e % 4 < drop ? 0.0f : v[set][e];
    }
    __device__ __forceinline__ void put(int u, char *planes, int set = 0) const {
        const float(&x)[E] = v[set];
        char *to = planes + (KC ? lds[0] + u * (THREADS * 4 / STAGE) * 16 : lds[KC ? 0 : u]);
        if constexpr (HALF) {
            const Halves s = split4_half({x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]}, scale[u]);
#pragma unroll
            for (int c = 0; c < 2; ++c) *reinterpret_cast<u32x2 *>(to + c * kPart) = s.p[c];
        } else {
            const Parts s = split4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
#pragma unroll
            for (int c = 0; c < 3; ++c) *reinterpret_cast<u32x2 *>(to + c * kPart) = s.p[c];
        }
    }
};

// `length` k in stages of STAGE, at least one: where K ends inside the last one, that one is the
// last STAGE k there are, of which the first `drop` were summed before and are
// zero in A.  Past the end it is loaded again and not used.
template <int STAGE>
struct Stages {
    int length, count, drop;
    __device__ __forceinline__ explicit Stages(int n)
        : length(n), count((n + STAGE - 1) / STAGE), drop(count * STAGE - n) {}
    __device__ __forceinline__ int start(int s) const { return min(s * STAGE, length - STAGE); }
    __device__ __forceinline__ bool cuts(int s) const { return s == count - 1 && drop > 0; }
};

// stage(i, s) for every s, i = s % TURN as a constant.
template <int TURN, class F>
__device__ __forceinline__ void turns(int stages, F stage) {
    static_assert(TURN == 2 || TURN == 4, "");
    constexpr std::integral_constant<int, 0> i0;
    constexpr std::integral_constant<int, 1> i1;
    constexpr std::integral_constant<int, 2 % TURN> i2;
    constexpr std::integral_constant<int, 3 % TURN> i3;
    int s = 0;
    for (; s + TURN <= stages; s += TURN) {
        stage(i0, s), stage(i1, s + 1);
        if constexpr (TURN == 4) stage(i2, s + 2), stage(i3, s + 3);
    }
    if (s < stages) {
        stage(i0, s);
        if constexpr (TURN == 4)
            if (s + 1 < stages) {
                stage(i1, s + 1);
                if (s + 2 < stages) stage(i2, s + 2);
            }
    }
}

// Tiles of a CU, for the registers that a wavefront may take.
constexpr int per_cu(int fm) { return fm == 4 ? 1 : fm == 2 ? 2 : 3; }

// What a tile of a workgroup takes of LDS.
template <int WM, int WN, int FM>
struct Room {
    using T = Tile<WM, WN, FM>;
    static constexpr int BM = T::BM, BN = T::BN;
    static constexpr bool kHalf = T::kHalf;
    static constexpr int kA = plane(BM, kStage), kB = plane(BN, kStage);                      // of 16 k
    static constexpr int kLongA = plane(BM, 2 * kStage), kLongB = plane(BN, 2 * kStage);      // of 32 k
    static constexpr int kPlanesA = 3 * 2 * kA, kBuffer = kPlanesA + 3 * 2 * kB;
    static constexpr int kHalfA = 2 * 4 * kLongA, kHalfBuffer = kHalfA + 2 * 4 * kLongB;
    static constexpr int kRowOut = 68;  // floats: 64 of a row of results, 16 bytes apart from the next one's banks
    static_assert(kBuffer >= (BM + BN) * kStage * 4, "");
    static_assert(2 * kBuffer >= T::kWaves * 32 * kRowOut * 4, "");
    alignas(128) char memory[2 * (kHalf ? kHalfBuffer : kBuffer)];
    int exponents[kHalf ? BM + BN : 1];
    float worst[kHalf ? 2 * T::kWaves : 1];
};

// Tile `id` of p's slices' tiles, `len` k a slice.
template <int WM, int WN, int FM, bool TA, bool TB>
__device__ __forceinline__ void one_tile(const Product &p, int tiles_m, int tiles_n, int64_t id, int len,
                                         Room<WM, WN, FM> &room) {
    using T = Tile<WM, WN, FM>;
    using R = Room<WM, WN, FM>;
    constexpr int BM = T::BM, BN = T::BN, kThreads = T::kThreads;
    constexpr bool kHalf = R::kHalf;
    constexpr int kA = R::kA, kB = R::kB, kLongA = R::kLongA, kLongB = R::kLongB;
    constexpr int kPlanesA = R::kPlanesA, kBuffer = R::kBuffer, kHalfA = R::kHalfA, kHalfBuffer = R::kHalfBuffer;
    constexpr int kRowOut = R::kRowOut;
    char(&memory)[sizeof(room.memory)] = room.memory;
    auto &exponents = room.exponents;
    auto &worst = room.worst;
    auto &xs = *reinterpret_cast<float(*)[kStage][BM]>(memory);
    auto &ys = *reinterpret_cast<float(*)[kStage][BN]>(memory + BM * kStage * 4);

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    const int64_t per = static_cast<int64_t>(tiles_m) * tiles_n;
    const int64_t slice = id / per, b = slice / p.splits;
    int tm, tn;
    grouped_tile(static_cast<int>(id - slice * per), tiles_m, tiles_n, 8, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int k0 = static_cast<int>(slice - b * p.splits) * len;
    const int k1 = max(k0, static_cast<int>(min(static_cast<int64_t>(k0) + len, static_cast<int64_t>(p.K))));
    const float *A = p.a.p + b * p.a.stride + (TA ? m0 : m0 * p.a.ld);
    const float *B = p.b.p + b * p.b.stride + (TB ? n0 * p.b.ld : n0);
    const int rows = p.M - m0, cols = p.N - n0;

    f32x16 acc[FM][2];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) acc[i][f] = f32x16{};
    };

    // FP32 multiplies: any shape, any value, one stage at a time.
    auto general = [&](int first, int last, const int64_t *skip) {
        for (int k = first; k < last; k += kStage) {
            __syncthreads();
#pragma unroll 1
            for (int o = tid; o < BM * kStage; o += kThreads) {
                const int r = TA ? o % BM : o / kStage, q = TA ? o / BM : o % kStage;
                float v = element<!TA>(A, p.a.ld, r, rows, k + q, last);
                if (skip != nullptr && k + q < last && skip[k + q] == p.ignore) v = 0.0f;
                xs[q][place_of_row(r)] = v;
            }
#pragma unroll 1
            for (int o = tid; o < BN * kStage; o += kThreads) {
                const int r = TB ? o / kStage : o % BN, q = TB ? o % kStage : o / BN;
                float v = element<TB>(B, p.b.ld, r, cols, k + q, last);
                if (skip != nullptr && k + q < last && skip[k + q] == p.ignore) v = 0.0f;
                ys[q][place_of_row(r)] = v;
            }
            __syncthreads();
#pragma unroll 2
            for (int q = 0; q < kStage; q += 2) {
                float y[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) y[f] = ys[q + half][64 * wn + 32 * f + col];
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const float x = xs[q + half][32 * (FM * wm + i) + col];
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y[f], acc[i][f], 0, 0, 0);
                }
            }
        }
        __syncthreads();
    };

    // The stages on the bf16 units.  A stage runs in 6 phases, a part of A
    // times a part of B each.  Under a phase's products the next phase's
    // operands are read from LDS, and the next stage's values, loaded into registers a
    // stage ago, are split and written to the other buffer and their
    // registers loaded again.  The one barrier lies before the last phase, under
    // which the next stage's first operands are read.
    auto quick = [&](int first, auto last) {
        Share<BM, kThreads, !TA, kStage, false> sa(A + (TA ? first * p.a.ld : first), p.a.ld, rows, m0 > 0, tid, nullptr);
        Share<BN, kThreads, TB, kStage, false> sb(B + (TB ? first : first * p.b.ld), p.b.ld, cols, n0 > 0, tid, nullptr);
        constexpr int kUa = decltype(sa)::kUnits, kUb = decltype(sb)::kUnits;
        const Stages<kStage> all(last - first);
        const int stages = all.count;
        u32x4 x[2][FM], y[3][2];  // parts of A by turns; the parts of B
        const int ra = half * kA + (32 * FM * wm + col) * 16;
        const int rb = kPlanesA + half * kB + (64 * wn + col) * 16;
        auto fetch_a = [&](int set, int part, const char *from) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                x[set][i] = *reinterpret_cast<const u32x4 *>(from + part * (2 * kA) + ra + 32 * 16 * i);
        };
        auto fetch_b = [&](int part, const char *from) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
                y[part][f] = *reinterpret_cast<const u32x4 *>(from + part * (2 * kB) + rb + 32 * 16 * f);
        };
        auto multiply = [&](int set, int part) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int f = i & 1 ? 1 - k : k;
                    acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, x[set][i]), __builtin_bit_cast(bf16x8, y[part][f]), acc[i][f], 0, 0, 0);
                }
            // between two matrix instructions: an LDS read, some of the
            // splitting, and its writes and loads
#pragma unroll
            for (int k = 0; k < FM * 2; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
            // the sums so far are used here, so their instructions stay ahead
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) asm volatile("" : "+v"(acc[i][f]));
            __builtin_amdgcn_sched_barrier(0);
        };
        // Set P of x holds l of A at the start, 1 - P at the end.
        auto stage = [&](auto pc, int s, const char *from, char *to) {
            constexpr int P = decltype(pc)::value, Q = 1 - P;
            const int next = all.start(s + 2);
            if (all.cuts(s + 1)) sa.cut(all.drop, tid);
            fetch_a(Q, 1, from);
            sa.put(0, to);
            multiply(P, 0);  // l h
            fetch_b(1, from);
            if constexpr (kUa > 1) sa.put(1, to);
            sa.load(next);
            multiply(Q, 0);  // m h
            fetch_a(P, 0, from);
            sb.put(0, to + kPlanesA);
            multiply(Q, 1);  // m m
            fetch_b(2, from);
            if constexpr (kUb > 1) sb.put(1, to + kPlanesA);
            sb.load(next);
            multiply(P, 1);  // h m
            multiply(P, 0);  // h h
            wait_older<63>();  // LDS accesses alone
            barrier_only();
            fetch_a(Q, 2, to);
            fetch_b(0, to);
            multiply(P, 2);  // h l
        };
        constexpr std::integral_constant<int, 0> p0;
        constexpr std::integral_constant<int, 1> p1;
        char *even = memory, *odd = memory + kBuffer;
        sa.load(0), sb.load(0);
#pragma unroll
        for (int u = 0; u < kUa; ++u) sa.put(u, even);
#pragma unroll
        for (int u = 0; u < kUb; ++u) sb.put(u, even + kPlanesA);
        sa.load(all.start(1)), sb.load(all.start(1));
        wait_older<63>();
        barrier_only();
        fetch_a(0, 2, even);
        fetch_b(0, even);
        int s = 0;
        for (; s + 1 < stages; s += 2) {
            stage(p0, s, even, odd);
            stage(p1, s + 1, odd, even);
        }
        if (s < stages) stage(p0, s, even, odd);
    };

    // Whether two fp16 parts do: the rows' exponents for scaling, and a bound.
    // Parts of a value are off by 2^-23 of it, or 2^-40 of a power of two above its row's
    // largest (and the product of two second parts, 2^-22 of the values' at most, is left out).
    // The latter adds up to less than n 2^-39 a b over the n products of a cell that
    // aren't zero, a and b those powers of two for its row and column; and the sum S
    // of their |a b| is at least n a b 2^-c with c the mean over them of
    // log2(a / |a_k|) + log2(b / |b_k|), as an arithmetic mean is at least the
    // geometric one.  With costs (that mean over all k, zeros counting nothing)
    // Ca and Cb and shares fa and fb of values that aren't zero, n is at least (fa
    // + fb - 1) K and c at most (Ca + Cb) / (fa + fb - 1).  Where c <= 17 for
    // the worst row with the worst column, all of it is below 2^-22 S.
    auto certified = [&]() {
        if constexpr (!kHalf) return false;
        static_assert(!kHalf || BM + BN == kThreads, "");
        const bool second = tid >= BM;
        const int r = second ? tid - BM : tid, count = second ? p.N : p.M;
        const int blocks = second ? p.blocks_b : p.blocks_a;
        const int64_t line = p.batch * count;
        const RowStat *from = (second ? p.row_b : p.row_a) + b * count + (second ? n0 : m0) + r;
        float cost = 0.0f, share = 1.0f;
        int e = 141;
        if (r < (second ? cols : rows)) {
            RowStat s{0, 0, 0, 0};
#pragma unroll 4
            for (int q = 0; q < blocks; ++q) {
                const RowStat t = from[q * line];
                s.top = max(s.top, t.top), s.count += t.count, s.sum += t.sum;
            }
            if (s.count > 0) {  // a row of zeros is one whatever its scale
                e = s.top;
                const float n = static_cast<float>(p.K);
                cost = (static_cast<float>(s.count) * static_cast<float>(e + 1) - static_cast<float>(s.sum)) / n;
                share = static_cast<float>(s.count) / n;
                if (e < 14 || e > 254) cost = __builtin_inff(), e = 141;
            }
        }
        exponents[tid] = e;
        for (int d = 1; d < 64; d *= 2) cost = fmaxf(cost, __shfl_xor(cost, d)), share = fminf(share, __shfl_xor(share, d));
        if (lane == 0) worst[2 * wave] = cost, worst[2 * wave + 1] = share;
        __syncthreads();
        float ca = 0.0f, cb = 0.0f, fa = 1.0f, fb = 1.0f;
        for (int w = 0; w < T::kWaves; ++w)
            if (w < BM / 64) ca = fmaxf(ca, worst[2 * w]), fa = fminf(fa, worst[2 * w + 1]);
            else cb = fmaxf(cb, worst[2 * w]), fb = fminf(fb, worst[2 * w + 1]);
        const float both = fa + fb - 1.0f;
        return both > 0.0f && ca + cb <= 17.0f * both;
    };
    // Back to the operands' scale.
    auto unscale = [&]() {
        const int en0 = exponents[BM + 64 * wn + 4 * (col & 15) + 2 * (col >> 4)];
        const int en1 = exponents[BM + 64 * wn + 4 * (col & 15) + 2 * (col >> 4) + 1];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int em = exponents[row_at(32 * (FM * wm + i) + (r & 3) + 8 * (r >> 2) + 4 * half)] - 282;
                acc[i][0][r] = ldexpf(acc[i][0][r], em + en0);
                acc[i][1][r] = ldexpf(acc[i][1][r], em + en1);
            }
    };
    // The small tiles' stages in bf16 parts: too few products a phase to
    // hide an LDS read, so a stage's operands are all read a stage ahead.
    // Under the products of stage s the operands of s + 1 are read from LDS, and the values
    // of s + 2 are split and written where those of s were.
    auto quick_small = [&](int first, int last) {
        // Stages that loads run ahead: four (both transposed, four spill: 54 x 2720 x 13019
        // 51.5 us, two 51.2) where a tile has registers for them.
        constexpr int D = FM == 1 && !(TA && TB) ? 4 : 2;
        Share<BM, kThreads, !TA, kStage, false, D> sa(A + (TA ? first * p.a.ld : first), p.a.ld, rows, m0 > 0, tid, nullptr);
        Share<BN, kThreads, TB, kStage, false, D> sb(B + (TB ? first : first * p.b.ld), p.b.ld, cols, n0 > 0, tid, nullptr);
        constexpr int kUa = decltype(sa)::kUnits, kUb = decltype(sb)::kUnits;
        const Stages<kStage> all(last - first);
        u32x4 x[2][3][FM], y[2][3][2];
        const int ra = half * kA + (32 * FM * wm + col) * 16;
        const int rb = kPlanesA + half * kB + (64 * wn + col) * 16;
        auto fetch = [&](int set, const char *from) {
#pragma unroll
            for (int c = 2; c >= 0; --c) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    x[set][c][i] = *reinterpret_cast<const u32x4 *>(from + c * (2 * kA) + ra + 32 * 16 * i);
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    y[set][c][f] = *reinterpret_cast<const u32x4 *>(from + c * (2 * kB) + rb + 32 * 16 * f);
            }
        };
        auto multiply = [&](int set, int ca, int cb) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, x[set][ca][i]), __builtin_bit_cast(bf16x8, y[set][cb][f]), acc[i][f], 0, 0, 0);
        };
        auto put = [&](char *to, int set) {
#pragma unroll
            for (int u = 0; u < kUa; ++u) sa.put(u, to, set);
#pragma unroll
            for (int u = 0; u < kUb; ++u) sb.put(u, to + kPlanesA, set);
        };
        auto load = [&](int s, int set) { sa.load(all.start(s), set), sb.load(all.start(s), set); };
        auto stage = [&](auto ic, int s) {
            constexpr int I = decltype(ic)::value, P = I % 2, S = (I + 2) % D;
            if (all.cuts(s + 2)) sa.cut(all.drop, tid, S);
            fetch(1 - P, memory + (1 - P) * kBuffer);
            put(memory + P * kBuffer, S);
            load(s + 2 + D, S);
            multiply(P, 2, 0), multiply(P, 0, 2), multiply(P, 1, 1);
            multiply(P, 1, 0), multiply(P, 0, 1), multiply(P, 0, 0);
#pragma unroll
            for (int k = 0; k < 6 * FM * 2; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) asm volatile("" : "+v"(acc[i][f]));
            wait_older<63>();  // LDS accesses alone
            barrier_only();
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, d);
        put(memory, 0);
        load(D, 0);
        if (all.cuts(1)) sa.cut(all.drop, tid, 1);
        put(memory + kBuffer, 1);
        load(D + 1, 1);
        wait_older<63>();
        barrier_only();
        fetch(0, memory);
        wait_older<63>();
        barrier_only();
        turns<D>(all.count, stage);
    };

    // Stages of 32 k in fp16 parts, as above: per 16 k the products l h,
    // h h and h l.
    auto quick_half = [&](int first, auto last) {
        constexpr int kLong = 2 * kStage;
        Share<BM, kThreads, !TA, kLong, true> sa(A + (TA ? first * p.a.ld : first), p.a.ld, rows, m0 > 0, tid, exponents);
        Share<BN, kThreads, TB, kLong, true> sb(B + (TB ? first : first * p.b.ld), p.b.ld, cols, n0 > 0, tid, exponents + BM);
        constexpr int kUa = decltype(sa)::kUnits, kUb = decltype(sb)::kUnits;
        static_assert(kUa == 4 && kUb == 4, "");
        const Stages<kLong> all(last - first);
        const int stages = all.count;
        u32x4 x[2][FM], y[3][2];
        const int ra = half * kLongA + (32 * FM * wm + col) * 16;
        const int rb = kHalfA + half * kLongB + (64 * wn + col) * 16;
        auto fetch_a = [&](int set, int part, int ks, const char *from) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                x[set][i] = *reinterpret_cast<const u32x4 *>(from + (part * 4 + 2 * ks) * kLongA + ra + 32 * 16 * i);
        };
        auto fetch_b = [&](int set, int part, int ks, const char *from) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
                y[set][f] = *reinterpret_cast<const u32x4 *>(from + (part * 4 + 2 * ks) * kLongB + rb + 32 * 16 * f);
        };
        auto multiply = [&](int sx, int sy) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int f = i & 1 ? 1 - k : k;
                    acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        __builtin_bit_cast(half8v, x[sx][i]), __builtin_bit_cast(half8v, y[sy][f]), acc[i][f], 0, 0, 0);
                }
#pragma unroll
            for (int k = 0; k < FM * 2; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) asm volatile("" : "+v"(acc[i][f]));
            __builtin_amdgcn_sched_barrier(0);
        };
        auto stage = [&](int s, const char *from, char *to) {
            const int next = all.start(s + 2);
            if (all.cuts(s + 1)) sa.cut(all.drop, tid);
            fetch_a(1, 0, 0, from);
            sa.put(0, to), sa.put(1, to);
            multiply(0, 0);  // l h
            fetch_b(1, 1, 0, from);
            sa.put(2, to), sa.put(3, to);
            sa.load(next);
            multiply(1, 0);  // h h
            fetch_a(0, 1, 1, from);
            fetch_b(2, 0, 1, from);
            sb.put(0, to + kHalfA), sb.put(1, to + kHalfA);
            multiply(1, 1);  // h l
            fetch_a(1, 0, 1, from);
            sb.put(2, to + kHalfA), sb.put(3, to + kHalfA);
            sb.load(next);
            multiply(0, 2);  // l h
            fetch_b(1, 1, 1, from);
            multiply(1, 2);  // h h
            wait_older<63>();
            barrier_only();
            fetch_a(0, 1, 0, to);
            fetch_b(0, 0, 0, to);
            multiply(1, 1);  // h l
        };
        char *even = memory, *odd = memory + kHalfBuffer;
        sa.load(0), sb.load(0);
#pragma unroll
        for (int u = 0; u < 4; ++u) sa.put(u, even), sb.put(u, even + kHalfA);
        sa.load(all.start(1)), sb.load(all.start(1));
        wait_older<63>();
        barrier_only();
        fetch_a(0, 1, 0, even);
        fetch_b(0, 0, 0, even);
        int s = 0;
        for (; s + 1 < stages; s += 2) {
            stage(s, even, odd);
            stage(s + 1, odd, even);
        }
        if (s < stages) stage(s, even, odd);
        unscale();
    };

    // The results of a block of 32 x 64 by way of LDS, so that a lane has 4
    // neighbouring columns of a row and the code below is there once: `use` gets
    // the row and column of the tile and the 4 values.
    float *out = reinterpret_cast<float *>(memory) + wave * 32 * kRowOut;
    auto each = [&](auto use) {
#pragma unroll 1
        for (int i = 0; i < FM; ++i) {
            auto dump = [&](auto ic) {
                constexpr int I = decltype(ic)::value;
                if constexpr (I < FM)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        *reinterpret_cast<f32x2 *>(out + ((r & 3) + 8 * (r >> 2) + 4 * half) * kRowOut +
                                                   4 * (col & 15) + 2 * (col >> 4)) = f32x2{acc[I][0][r], acc[I][1][r]};
            };
            if (i == 0) dump(std::integral_constant<int, 0>{});
            if (i == 1) dump(std::integral_constant<int, 1>{});
            if (i == 2) dump(std::integral_constant<int, 2>{});
            if (i == 3) dump(std::integral_constant<int, 3>{});
            wait_older<63>();
#pragma unroll 1
            for (int q = lane >> 4; q < 32; q += 4)
                use(row_at(32 * (FM * wm + i) + q), 64 * wn + 4 * (lane & 15),
                    *reinterpret_cast<const f32x4 *>(out + q * kRowOut + 4 * (lane & 15)));
            wait_older<63>();
        }
    };
    // Whether a sum that counts is infinite or NaN (an infinity's parts are NaN).
    auto odd = [&]() {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int r = 0; r < 16; ++r) t = fmaf(acc[i][f][r], 0.0f, t);
        bool found = false;
        if (__ballot(t != 0.0f))  // NaN too
            each([&](int r, int c, f32x4 v) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r < rows && c + e < cols && !finite(v[e]) && (p.mode == kStore || p.target[m0 + r] != p.ignore))
                        found = true;
            });
        return found;
    };

    clear();
    int whole = k0;  // the end of what the stages take
    bool check = false;
    if (p.narrow) {
        bool half_parts = false;
        if constexpr (kHalf)
            if (p.row_b != nullptr && k1 - k0 >= 2 * kStage && certified()) {
                quick_half(k0, k1);
                whole = k1;
                half_parts = true;
            }
        if (!half_parts && k1 - k0 >= kStage) {
            whole = k1;
            check = true;
            if constexpr (FM == 4)
                quick(k0, k1);
            else
                quick_small(k0, k1);
        }
    }
    for (int from = whole;; from = k0) {
        if (from < k1) general(from, k1, p.target_k);
        if (!check) break;
        check = false;
        if (!__syncthreads_or(odd())) break;
        clear();
    }
    __syncthreads();

    // ---- results ----
    auto put = [&](float *dst, int c, f32x4 v) {
        if (c + 3 < cols) {
            *reinterpret_cast<float4u *>(dst + c) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (c + e < cols) dst[c + e] = v[e];
        }
    };
    auto get = [&](const float *src, int c) {
        f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
        if (c + 3 < cols) {
            v = *reinterpret_cast<const float4u *>(src + c);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (c + e < cols) v[e] = src[c + e];
        }
        return v;
    };
    if (p.mode >= kStats) {
        const bool fine = p.M <= kFineTokens;
        const int lanes = fine ? 4 : 16;  // that share a piece of a row
        each([&](int r, int c, f32x4 v) {
            float top = -__builtin_inff(), s = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = c + e < cols ? fmaxf(top, v[e]) : top;
            auto larger = [](float a, float b) { return fmaxf(a, b); };
            top = fine ? over_lanes<4>(top, larger) : over_lanes<16>(top, larger);
            const float base = base_of(top);
#pragma unroll
            for (int e = 0; e < 4; ++e) s += c + e < cols ? quick_exp(v[e] - base) : 0.0f;
            auto sum = [](float a, float b) { return a + b; };
            s = fine ? over_lanes<4>(s, sum) : over_lanes<16>(s, sum);
            if (r < rows && c < cols) {
                const int64_t m = m0 + r;
                if ((lane & (lanes - 1)) == 0) p.stats[m * p.groups + (n0 + c) / (4 * lanes)] = stat2{top, s};
                const int64_t t = p.target[m] - n0 - c;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t == e && c + e < cols) p.at_target[m] = v[e];
                if (p.mode == kStoreStats) put(p.c.p + m * p.c.ld + n0, c, v);
            }
        });
    } else if (p.splits > 1) {
        float *W = p.slices + (slice * p.M + m0) * p.N + n0;
        each([&](int r, int c, f32x4 v) {
            if (r < rows && c < cols) put(W + static_cast<int64_t>(r) * p.N, c, v);
        });
    } else {
        float *C = p.c.p + b * p.c.stride + m0 * p.c.ld + n0;
        float *Z = p.e.pre.p != nullptr ? p.e.pre.p + b * p.e.pre.stride + m0 * p.e.pre.ld + n0 : nullptr;
        const float *R = p.e.residual.p != nullptr ? p.e.residual.p + b * p.e.residual.stride + m0 * p.e.residual.ld + n0
                                                   : nullptr;
        const int c = 64 * wn + 4 * (lane & 15);
        const f32x4 bias = p.e.bias.p != nullptr ? get(p.e.bias.p + b * p.e.bias.stride + n0, c)
                                                 : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        each([&](int r, int, f32x4 v) {
            if (r >= rows || c >= cols) return;
            if (p.mode == kStoreSome && p.target[m0 + r] == p.ignore) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (p.e.bias.p != nullptr) v += bias;
            if (Z != nullptr) put(Z + r * p.e.pre.ld, c, v);
            if (p.e.activation != GEMM_F32_ACT_NONE)
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    const float y = activate(p.e.activation, v[0]);
                    v = f32x4{v[1], v[2], v[3], y};
                }
            if (R != nullptr) v += get(R + r * p.e.residual.ld, c);
            put(C + r * p.c.ld, c, v);
        });
    }
}

template <int WM, int WN, int FM, bool TA, bool TB>
__global__ __launch_bounds__(64 * WM * WN, per_cu(FM)) void tile_kernel(Product p, int tiles_m, int tiles_n,
                                                                        int64_t first_tile, int len) {
    __shared__ Room<WM, WN, FM> room;
    one_tile<WM, WN, FM, TA, TB>(p, tiles_m, tiles_n, first_tile + xcd_remap(blockIdx.x, gridDim.x), len, room);
}

// Tiles of a product, and whole stages a slice.
struct TileGrid {
    int tiles_m, tiles_n, len;
    int64_t tiles;
};
template <int WM, int WN, int FM>
TileGrid tile_grid(const Product &p) {
    using T = Tile<WM, WN, FM>;
    constexpr int kWhole = T::kHalf ? 2 * kStage : kStage;
    TileGrid g{static_cast<int>(div_up(p.M, T::BM)), static_cast<int>(div_up(p.N, T::BN)),
               static_cast<int>(div_up(div_up(p.K, kWhole), p.splits)) * kWhole, 0};
    g.tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n * p.batch * p.splits;
    return g;
}

template <int WM, int WN, int FM, bool TA, bool TB>
hipError_t launch_one(const Product &p, hipStream_t stream) {
    const TileGrid g = tile_grid<WM, WN, FM>(p);
    for (int64_t t = 0; t < g.tiles; t += 1 << 21) {  // (a launch's threads are counted in 32 bits)
        const unsigned grid = static_cast<unsigned>(std::min<int64_t>(g.tiles - t, 1 << 21));
        tile_kernel<WM, WN, FM, TA, TB><<<grid, 64 * WM * WN, 0, stream>>>(p, g.tiles_m, g.tiles_n, t, g.len);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <bool TA, bool TB>
hipError_t launch_tile(const Product &p, int tile, hipStream_t stream) {
    return tile == 0   ? launch_one<2, 4, 4, TA, TB>(p, stream)
           : tile == 1 ? launch_one<2, 2, 2, TA, TB>(p, stream)
                       : launch_one<2, 2, 1, TA, TB>(p, stream);
}

}  // namespace fused
}  // namespace gemm_f32_impl
