// C = A B^T with both operands in MXFP4 (include/gemm_mxfp4.h).

#include <algorithm>
#include <type_traits>

#include "mxfp4.h"
#include "mxfp4_device.h"

namespace gemm_f32_impl {
namespace mx {
namespace {

// acc += X Y over one 32 x 32 x 64 step; T selects the byte of the scale words.
template <int T>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 x, u32x4 y, f32x16 acc, uint32_t ex, uint32_t ey) {
    const i32x8 X = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    const i32x8 Y = {(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(X, Y, acc, 4, 4, T, (int)ex, T, (int)ey);
}

// A tile of WM x WN wavefronts, each FM x FN blocks of 32 x 32.  K runs in
// stages of 128 (4 blocks of every row), kStages of them (a group: 512 k) in
// LDS at a time.
template <int FM, int FN, int WM, int WN>
struct Tile {
    static constexpr int BM = FM * WM * 32, BN = FN * WN * 32, R = BM + BN, NW = WM * WN;
    static constexpr int kStages = 4, kStageBlocks = 4, kRowBytes = 2 * kStageBlocks * kBlockBytes;
    static constexpr int kGroupBlocks = kStages * kStageBlocks;
    static constexpr int kLoads = R / 8 / NW;                    // a wavefront's code loads per two stages
    static constexpr int kScaleLoads = (R / 64 + NW - 1) / NW;   // ... scale loads per group
    static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0, "");
};

// Persistent kernel: a workgroup walks over tiles, and its loads run one
// group ahead of its products, over the ends of tiles too.
//
// In v_mfma_scale_f32_32x32x64_f8f6f4 lane l holds the codes of row l % 32,
// block l / 32 of two, and that block's scale.  Which two blocks meet in one
// instruction is free as long as A and B agree: in a stage, lanes 0-31 take
// blocks 0 and 1, lanes 32-63 blocks 2 and 3, so a lane's scales are one half
// of the row's scale word.
//
// LDS holds two stages of a row as 8 slots of 16 bytes, filled by direct
// loads (64 lanes x 16 bytes into 1 KiB: 8 rows).  That is a line of the
// caches: loaded a stage at a time, half a line each, L2 had twice the
// requests, three quarters of what its channels answer (1024 x 1024 x 65536:
// 53 us so, 46 with whole lines; 4096^3: 49 and 46).  Block b of row r sits in
// slot b ^ (r / 2 % 8): 16 lanes that read one block of 16 rows then touch
// every bank once.
//
// Order within a stage: the fragments of its second half are read under the
// products of its first.  In every second stage a barrier follows, after
// which the next two stages are in LDS and these ones' buffer is free, and
// the loads one group on go out under the products of the second half, as in
// every stage the next one's first fragments.  So neither the barrier nor an
// LDS read is waited for with idle matrix cores.
// A CU holds PER_CU workgroups, which gives every SIMD two wavefronts: with
// one (4 x 4 blocks each) it idles wherever that one waits, and 8192 x 14336 x
// 4096 took 293 us instead of 276 (with half lines).
//
// 8192 x 14336 x 4096 takes 255 to 284 us by card on the codes of normal
// values (3.4 to 3.8 PFLOP/s) and a little longer on random ones.  A loop of
// nothing but these instructions on random codes reaches 5.5, where the card's
// power holds its clock; of the rest, storing C is little: half the results of
// as many products (4096 x 14336 x 8192) take 4% less, and workgroups that
// start at different times, so that some store while others multiply, gain 3%.
//
// 1024 x 1024 x 65536 on 128 x 128 tiles (46 to 48 us) fills no one unit: of a
// CU's 81,000 cycles the path on which loads return is busy 66,000 (in 26,000 of
// them it waits for L1 or L2), the one of their addresses 50,000, the matrix
// cores 33,000 and LDS reads 22,000.  The codes alone need 33,000 cycles of the
// first at the 64 bytes a cycle that L1 gives; a third of all requests are the
// 16 bytes of scales a row and group, a line of L1 each.
template <int FM, int FN, int WM, int WN, int PER_CU, bool WHOLE>
__global__ __launch_bounds__(WM *WN * 64, PER_CU *WM *WN / 4) void product_tile_kernel(Product p, int tiles_m,
                                                                        int tiles_n, int64_t tiles,
                                                                        int groups, int len) {
    using T = Tile<FM, FN, WM, WN>;
    __shared__ __align__(1024) uint8_t codes0[T::R * T::kRowBytes];  // stages 0 and 1 of a group
    __shared__ __align__(1024) uint8_t codes1[T::R * T::kRowBytes];  // 2 and 3
    __shared__ __align__(1024) uint32_t scales[2 * T::kStages * T::R];  // [group parity][stage][row]

    const int lane = threadIdx.x & 63, half = lane >> 5, row = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int nb = (p.K + kBlock - 1) / kBlock, words = (nb + 3) / 4;
    const int64_t grid = gridDim.x;

    // ---- loads: codes one group ahead of the products, scales two ----
    struct Cursor {
        int64_t id;
        int g, g1;
        Rows a, b;
    };
    auto seek = [&](Cursor &c, bool scale) {  // to the start of tile c.id
        if (c.id >= tiles) {
            c.g = 0, c.g1 = 0;
            return;
        }
        const Place q = place_of<T::BM, T::BN>(p, c.id, tiles_m, tiles_n, groups, len);
        const int64_t b = q.slice / p.splits;
        c.g = q.g0, c.g1 = q.g1;
        if (scale) {
            c.a = rows_from(p.a.scales + b * p.a.ss, p.a.lds, q.m0, p.M, words * 4);
            c.b = rows_from(p.b.scales + b * p.b.ss, p.b.lds, q.n0, p.N, words * 4);
        } else {
            c.a = rows_from(p.a.codes + b * p.a.sq, p.a.ldq, q.m0, p.M, nb * kBlockBytes);
            c.b = rows_from(p.b.codes + b * p.b.sq, p.b.ldq, q.n0, p.N, nb * kBlockBytes);
        }
    };
    auto advance = [&](Cursor &c, bool scale) {
        if (++c.g >= c.g1) {
            c.id += grid;
            seek(c, scale);
        }
    };
    const int lrow = wave * 8 + (lane >> 3);                 // row of a lane's first load
    const int blk = (lane & 7) ^ ((lrow >> 1) & 7);          // block of its slot
    auto load = [&](const Cursor &c, int pair, uint8_t *codes) {
        const int block = c.g * T::kGroupBlocks + pair * 2 * T::kStageBlocks + blk;
        const int off = c.g < c.g1 ? min(block, nb - 1) * kBlockBytes : kOutside;
#pragma unroll
        for (int j = 0; j < T::kLoads; ++j) {
            const bool in_a = j * T::NW * 8 < T::BM;
            const Rows &m = in_a ? c.a : c.b;
            const int r = j * T::NW * 8 - (in_a ? 0 : T::BM);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(m.rsrc, (lptr_t)(codes + (j * T::NW + wave) * 1024),
                                                     16, (lrow + r) * m.ld + off, 0, 0, 0);
        }
    };
    // A group's scales, 16 bytes of a row per lane: the cache answers so many
    // requests a cycle, whatever they carry, and a word per row and stage was
    // two thirds of all requests.
    u32x4 held[T::kScaleLoads];
    auto fetch_scales = [&](const Cursor &c) {
#pragma unroll
        for (int j = 0; j < T::kScaleLoads; ++j) {
            const int r = (j * T::NW + wave) * 64;
            const Rows &m = r < T::BM ? c.a : c.b;
            const int at = (r - (r < T::BM ? 0 : T::BM) + lane) * m.ld;
            const int off = c.g < c.g1 && r < T::R ? 0 : kOutside;
            if constexpr (WHOLE) {
                held[j] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(m.rsrc, (at + 16 * c.g) | off, 0, 0));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    held[j][k] = __builtin_amdgcn_raw_buffer_load_b32(
                        m.rsrc, (at + 4 * min(4 * c.g + k, words - 1)) | off, 0, 0);
            }
        }
    };
    // Blocks past the end get scale 2^-127 on both sides: whatever their
    // codes, such products are below 2^-240 and leave an FP32 sum as it is.
    int put = lane;  // + group parity x 4 R
    auto store_scales = [&](int g) {
#pragma unroll
        for (int j = 0; j < T::kScaleLoads; ++j) {
            const int r = (j * T::NW + wave) * 64;
            if (T::R % (64 * T::NW) && r >= T::R) break;
#pragma unroll
            for (int k = 0; k < T::kStages; ++k) {
                const int valid = min(max(nb - (g * T::kStages + k) * T::kStageBlocks, 0), 4);
                const uint32_t mask = valid == 4 ? 0xffffffffu : (1u << (8 * valid)) - 1u;
                scales[put + k * T::R + r] = held[j][k] & mask;
            }
        }
        put = 2 * lane + 4 * T::R - put;
    };

    // ---- fragments ----
    // Byte offsets of the lane's two blocks in a stage.  Opaque values keep
    // the read addresses within reach of the compiler's alias analysis, which
    // else waits for the loads of other buffers first.
    const int ra = wm * FM * 32 + row, rb = T::BM + wn * FN * 32 + row;
    int oa[2], ob[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int slot = ((2 * half + t) ^ ((row >> 1) & 7)) * kBlockBytes;
        oa[t] = ra * T::kRowBytes + slot;
        ob[t] = rb * T::kRowBytes + slot;
        asm volatile("" : "+v"(oa[t]), "+v"(ob[t]));
    }
    // half words of the lane's scales, + group parity x 8 R (read_scales turns it first)
    int oea = 2 * ra + half + 8 * T::R, oeb = 2 * rb + half + 8 * T::R;
    asm volatile("" : "+v"(oea), "+v"(oeb), "+v"(put));
    u32x4 x[2][FM], y[2][FN];
    uint32_t ea[2][FM], eb[2][FN];  // [stage parity]
    auto fetch = [&](auto tc, const uint8_t *codes) {
        constexpr int t = decltype(tc)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            x[t][i] = *reinterpret_cast<const u32x4 *>(codes + oa[t] + 32 * i * T::kRowBytes);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            y[t][j] = *reinterpret_cast<const u32x4 *>(codes + ob[t] + 32 * j * T::kRowBytes);
        oa[t] ^= 4 * kBlockBytes, ob[t] ^= 4 * kBlockBytes;  // the other stage's
        asm volatile("" : "+v"(oa[t]), "+v"(ob[t]));
    };
    auto read_scales = [&](auto uc, int stage) {
        constexpr int u = decltype(uc)::value;
        const uint16_t *halves = reinterpret_cast<const uint16_t *>(scales);
        if (stage == 0) {  // the next group's
            oea = 4 * ra + 2 * half + 8 * T::R - oea;
            oeb = 4 * rb + 2 * half + 8 * T::R - oeb;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) ea[u][i] = halves[oea + 2 * (stage * T::R + 32 * i)];
#pragma unroll
        for (int j = 0; j < FN; ++j) eb[u][j] = halves[oeb + 2 * (stage * T::R + 32 * j)];
    };

    f32x16 acc[FM][FN];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    };
    auto multiply = [&](auto tc, auto uc) {
        constexpr int t = decltype(tc)::value, u = decltype(uc)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int k = 0; k < FN; ++k) {
                const int j = i & 1 ? FN - 1 - k : k;  // one operand stays from each to the next
                acc[i][j] = mfma_fp4<t>(x[t][i], y[t][j], acc[i][j], ea[u][i], eb[u][j]);
            }
    };
    // One load or LDS read between two matrix instructions: issued in a row
    // they would keep the matrix cores waiting.
    auto interleave = [&](int loads, int reads) {
#pragma unroll
        for (int k = 0; k < FM * FN; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (reads > FM * FN / 2 && 2 * k < reads)
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            else if (k < reads)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (loads > FM * FN && 2 * k < loads)
                __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
            else if (k < loads)
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        // The sums so far are used here, so their instructions stay ahead.
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) asm volatile("" ::"a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
    };

    // C is streamed past the caches, which hold A and B (64 products of 1024^3:
    // 86 us with ordinary stores, 76 so), if its rows are whole lines.  Else
    // blocks share lines, which L2 has to gather, and a row's blocks are stored
    // one after the other (8192 x 14335 x 4096: 459 us streamed, 337 with
    // ordinary stores block by block, 282 row by row).
    auto store_tile = [&](int64_t id) {
        const Place q = place_of<T::BM, T::BN>(p, id, tiles_m, tiles_n, groups, len);
        const int64_t ldc = p.splits > 1 ? p.N : p.ldc;
        const float *base = p.splits > 1 ? p.W + q.slice * p.M * ldc : p.C + q.slice * p.sc;
        const int mw = q.m0 + wm * FM * 32, nw = q.n0 + wn * FN * 32;
        if (mw >= p.M || nw >= p.N) return;  // nothing of C: the buffer below would have no bytes
        const __amdgpu_buffer_rsrc_t c =
            buffer_of(base + mw * ldc + nw, ((p.M - 1 - mw) * ldc + p.N - nw) * 4);
        const int ld = static_cast<int>(ldc) * 4;
        int at[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = 32 * j + row;
            at[j] = nw + n < p.N ? n * 4 + 4 * half * ld : kOutside;
        }
        auto store = [&](auto policy) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const float v = acc[i][j][r];  // (a bit cast of the element itself takes element 0)
                        __builtin_amdgcn_raw_buffer_store_b32(
                            __builtin_bit_cast(uint32_t, v), c,
                            at[j] + (32 * i + (r & 3) + 8 * (r >> 2)) * ld, 0, decltype(policy)::value);
                    }
        };
        if (ldc % 32 == 0 && reinterpret_cast<uintptr_t>(base) % 128 == 0)
            store(std::integral_constant<int, kStream>{});
        else
            store(std::integral_constant<int, 0>{});
    };

    std::integral_constant<int, 0> c0;
    std::integral_constant<int, 1> c1;

    // Consecutive tiles go to workgroups of one XCD.
    int64_t id = xcd_remap(blockIdx.x, gridDim.x);
    Cursor cc, cs;
    cc.id = cs.id = id;
    seek(cc, false);
    seek(cs, true);
    fetch_scales(cs);
    load(cc, 0, codes0);
    load(cc, 1, codes1);
    store_scales(cs.g);
    advance(cs, true);
    fetch_scales(cs);
    store_scales(cs.g);
    advance(cs, true);
    advance(cc, false);
    wait_older<0>();
    barrier_only();
    fetch(c0, codes0);
    read_scales(c0, 0);

    constexpr int L = T::kLoads, S = T::kScaleLoads * (WHOLE ? 1 : 4);
    // Stage `i` of the group: products from `cur`, the next stage in `nxt`.
    // The waits count on the order of loads: the scales (S) go out in stage 1
    // ahead of its barrier, the codes of two stages (L) behind those of stages
    // 1 and 3, each behind a scheduling barrier of its own, since the scheduler
    // may turn loads of one region around.  What follows stage 1 was loaded in
    // the last group's stage 3, and the scales alone are younger; what follows
    // stage 3 in this group's stage 1, and nothing is.
#define GEMM_MXFP4_STAGE(i, cur, nxt, u, v)                                          \
    fetch(c1, cur);                                                                  \
    read_scales(v, (i + 1) % 4);                                                     \
    if (i == 1) fetch_scales(cs);                                                    \
    multiply(c0, u);                                                                 \
    interleave(i == 1 ? S : 0, 2 * (FM + FN));                                       \
    if (i & 1) {                                                                     \
        wait_older<i == 1 ? S : 0>();                                                \
        barrier_only();                                                              \
        if (i == 3) store_scales(cs.g);                                              \
        load(cc, i / 2, cur);                                                        \
    }                                                                                \
    fetch(c0, nxt);                                                                  \
    multiply(c1, u);                                                                 \
    interleave(i & 1 ? L : 0, FM + FN);

    for (; id < tiles; id += grid) {
        const Place at = place_of<T::BM, T::BN>(p, id, tiles_m, tiles_n, groups, len);
        clear();
        for (int g = at.g0; g < at.g1; ++g) {
            GEMM_MXFP4_STAGE(0, codes0, codes0, c0, c1)
            GEMM_MXFP4_STAGE(1, codes0, codes1, c1, c0)
            GEMM_MXFP4_STAGE(2, codes1, codes1, c0, c1)
            GEMM_MXFP4_STAGE(3, codes1, codes0, c1, c0)
            advance(cc, false);
            advance(cs, true);
        }
        store_tile(id);
    }
#undef GEMM_MXFP4_STAGE
    wait_older<0>();  // no load may land in LDS after the workgroup has ended
}

// Few rows, and operands of any stride: a workgroup of NW wavefronts holds a
// tile of 32 x 32 NT, its wavefronts take steps of 256 k in turn, straight
// from global memory, and their sums are added in LDS in a fixed order.  What
// it waits for is memory: every lane has 64 consecutive bytes of a row of B
// (and A) on the way per step.  256^3 3.5 us, 1000 x 1023 x 777 6.8 us.
template <int NT, int NW>
__global__ __launch_bounds__(NW * 64) void product_rows_kernel(Product p, int64_t tiles_m,
                                                               int64_t tiles_n, int64_t tiles) {
    __shared__ __align__(16) float part[NW][NT][16][64];
    const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int nb = (p.K + kBlock - 1) / kBlock, words = (nb + 3) / 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t line = t / tiles_n, b = line / tiles_m;
        const int64_t n0 = (t - line * tiles_n) * 32 * NT, m0 = (line - b * tiles_m) * 32;
        const int64_t m = min(m0 + row, int64_t{p.M} - 1);
        const uint8_t *A = p.a.codes + b * p.a.sq + m * p.a.ldq;
        const uint8_t *As = p.a.scales + b * p.a.ss + m * p.a.lds;
        const uint8_t *B[NT], *Bs[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t n = min(n0 + 32 * j + row, int64_t{p.N} - 1);
            B[j] = p.b.codes + b * p.b.sq + n * p.b.ldq;
            Bs[j] = p.b.scales + b * p.b.ss + n * p.b.lds;
        }
        f32x16 acc[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = f32x16{};
        // lanes 0-31 take blocks 0-3 of a step, lanes 32-63 blocks 4-7: their
        // scales are one word.  Blocks past the end get scale 2^-127 on both
        // sides, which leaves an FP32 sum as it is.
        for (int s = wave; s * 8 < nb; s += NW) {
            const int first = s * 8 + 4 * half, valid = min(max(nb - first, 0), 4);
            const uint32_t mask = valid == 4 ? 0xffffffffu : (1u << (8 * valid)) - 1u;
            const int w = min(first / 4, words - 1) * 4;
            const uint32_t ea = *reinterpret_cast<const uint32_t *>(As + w) & mask;
            uint32_t eb[NT];
            u32x4 x[4], y[NT][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t off = min(first + k, nb - 1) * int64_t{kBlockBytes};
                x[k] = *reinterpret_cast<const u32x4 *>(A + off);
#pragma unroll
                for (int j = 0; j < NT; ++j) y[j][k] = *reinterpret_cast<const u32x4 *>(B[j] + off);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) eb[j] = *reinterpret_cast<const uint32_t *>(Bs[j] + w) & mask;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[j] = mfma_fp4<0>(x[0], y[j][0], acc[j], ea, eb[j]);
                acc[j] = mfma_fp4<1>(x[1], y[j][1], acc[j], ea, eb[j]);
                acc[j] = mfma_fp4<2>(x[2], y[j][2], acc[j], ea, eb[j]);
                acc[j] = mfma_fp4<3>(x[3], y[j][3], acc[j], ea, eb[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) part[wave][j][r][lane] = acc[j][r];
        __syncthreads();
        for (int e = threadIdx.x; e < NT * 1024; e += NW * 64) {
            const int l = e & 63, r = (e >> 6) & 15, j = e >> 10;
            const int64_t n = n0 + 32 * j + (l & 31), mm = m0 + (r & 3) + 8 * (r >> 2) + 4 * (l >> 5);
            if (mm >= p.M || n >= p.N) continue;
            float v = part[0][j][r][l];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += part[w][j][r][l];
            p.C[b * p.sc + mm * p.ldc + n] = v;
        }
        __syncthreads();
    }
}

template <int NT, int NW>
hipError_t launch_rows(const Product &p, hipStream_t stream) {
    const int64_t tm = (p.M + int64_t{31}) / 32, tn = (p.N + int64_t{32 * NT - 1}) / (32 * NT);
    const int64_t tiles = tm * tn * p.batch;
    product_rows_kernel<NT, NW><<<static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 20)), NW * 64, 0,
                                  stream>>>(p, tm, tn, tiles);
    return hipGetLastError();
}

template <int FM, int FN, int WM, int WN, int PER_CU>
hipError_t launch_tile(const Product &p, hipStream_t stream) {
    using T = Tile<FM, FN, WM, WN>;
    const int tm = ceil_div(p.M, T::BM), tn = ceil_div(p.N, T::BN);
    const int64_t tiles = static_cast<int64_t>(tm) * tn * p.batch * p.splits;
    const int groups = ceil_div(static_cast<int>(blocks_of(p.K)), T::kGroupBlocks);
    const int len = ceil_div(groups, p.splits);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, 256 * PER_CU));
    if (groups * T::kStages * T::kStageBlocks == blocks_of(p.K))
        product_tile_kernel<FM, FN, WM, WN, PER_CU, true>
            <<<grid, T::NW * 64, 0, stream>>>(p, tm, tn, tiles, groups, len);
    else
        product_tile_kernel<FM, FN, WM, WN, PER_CU, false>
            <<<grid, T::NW * 64, 0, stream>>>(p, tm, tn, tiles, groups, len);
    return hipGetLastError();
}

// Partial sums of the slices of K, added in ascending order.  Where they are
// many and small, a load a time would be waited for a time (64 slices of 64 x
// 1024: 12 us less with 7 on the way); 8 of 1024 x 1024 take 8.3 to 9.3 us,
// 4.1 to 4.5 TB/s.
template <int V>
__global__ __launch_bounds__(256) void sum_slices_kernel(Product p, int64_t total) {
    typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
    const int64_t plane = static_cast<int64_t>(p.M) * p.N, per_row = p.N / V;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
         e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t line = e / per_row, j = (e - line * per_row) * V, b = line / p.M, i = line - b * p.M;
        const float *w = p.W + b * p.splits * plane + i * p.N + j;
        vec v = *reinterpret_cast<const vec *>(w);
        int s = 1;
        for (; s + 7 <= p.splits; s += 7) {  // 7 loads on the way
            vec u[7];
#pragma unroll
            for (int i = 0; i < 7; ++i) u[i] = *reinterpret_cast<const vec *>(w + (s + i) * plane);
#pragma unroll
            for (int i = 0; i < 7; ++i) v += u[i];
        }
        for (; s < p.splits; ++s) v += *reinterpret_cast<const vec *>(w + s * plane);
        *reinterpret_cast<vec *>(p.C + b * p.sc + i * p.ldc + j) = v;
    }
}

}  // namespace

int product_splits(int64_t batch, int64_t M, int64_t N, int64_t K) {
    return product_choice::choose(batch, M, N, K, kMostSplits).splits;
}

hipError_t launch_sum_slices(const Product &p, hipStream_t stream) {
    const int v = p.N % 4 == 0 ? 4 : 1;
    const int64_t total = p.batch * p.M * (p.N / v);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, 8192));
    if (v == 4)
        sum_slices_kernel<4><<<grid, 256, 0, stream>>>(p, total);
    else
        sum_slices_kernel<1><<<grid, 256, 0, stream>>>(p, total);
    return hipGetLastError();
}

hipError_t launch_product(const Product &asked, hipStream_t stream) {
    Product p = asked;
    using namespace product_choice;
    Choice c = choose(p.batch, p.M, p.N, p.K, p.splits > 1 ? kMostSplits : 1);
    if (!reaches(std::max({p.a.ldq, p.b.ldq, p.a.lds, p.b.lds}), std::max(p.ldc, int64_t{p.N}))) c = {kRows, 1};
    p.splits = c.splits;
    hipError_t err = hipSuccess;
    switch (c.kernel) {
        case kLarge: err = launch_tile<2, 4, 4, 2, 1>(p, stream); break;
        case kMedium: err = launch_tile<2, 2, 2, 2, 2>(p, stream); break;
        case kRows: err = launch_rows<1, 8>(p, stream); break;
    }
    if (err == hipSuccess && p.splits > 1) err = launch_sum_slices(p, stream);
    return err;
}

}  // namespace mx
}  // namespace gemm_f32_impl
