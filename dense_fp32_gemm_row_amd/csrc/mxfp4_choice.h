// Which kernel an MXFP4 product takes (host code alone; the tests ask it what
// their sizes run).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace gemm_f32_impl {
namespace mx {

constexpr int kBlock = 32;        // values that share a scale
constexpr int kBlockBytes = 16;   // their codes
constexpr int kMostSplits = 64;   // slices of K that a tile may be asked for

// Predicted microseconds of adding `splits` partial sums.
inline double sum_slices_us(double batch, double M, double N, int splits) {
    return splits > 1 ? 4.0 + batch * M * N * 4.0 * (splits + 1) / 3.5e6 : 0.0;
}

// Slices of K of `chunks` chunks each are equally long but for the last: with
// `want` asked for, the number that is not empty.
inline int slices_used(int64_t chunks, int64_t want) {
    const int64_t len = (chunks + want - 1) / want;
    return static_cast<int>((chunks + len - 1) / len);
}

inline int64_t blocks_of(int64_t k) { return (k + kBlock - 1) / kBlock; }

// ---- C = A B^T, both operands in the format ----
namespace product_choice {

// Which kernel a product takes: the least predicted time.  The figures are
// microseconds measured on MI355X, per 512 k of a tile and per store of one
// with the chip full, and for lone tiles:
//
//   256 x 256  5 + rounds (3.5 / 512 k + 10.8), one tile a CU; a lone tile
//              2.6 / 512 k
//   128 x 128  4 + rounds (2.35 / 512 k + 5), two tiles a CU; a lone tile
//              1.05 / 512 k
//   32 x 32    3 + 1 / 2048 k where there are few, up to 1.6 with a tile a CU
//              and 2.4 with 32 rows of A in it, 0.5 at least
//
// (Products of a few microseconds from a graph: called one by one they wait
// for their host.)  Over 253 products of up to 4e10 operations that leaves
// 0.03% on average and 7% at most to the better of 128 x 128 and 32 x 32.
//
// So 8192 x 14336 x 4096 (255 us, 284 on a slower card, against 318 with 128 x
// 128) and 64 x 1024^3 (66, on a slower card 88, against 80) take the large tile,
// 1024 x 1024 x 65536 128 x 128 with sliced K (46 and 8 for the sum, against 55
// and 8 with the large tile), 256^3 (2.9 against 5.9), 1000 x 1023 x 777 (6.0
// against 7.8) and products of few rows 32 x 32.
enum Kernel { kLarge, kMedium, kRows };
struct Choice {
    Kernel kernel;
    int splits;
};
inline double tile_us(int64_t tiles, double groups, int slots, double fixed, double each, double lone,
                      double store) {
    const double full = static_cast<double>(tiles / slots), rem = static_cast<double>(tiles % slots) / slots;
    double t = fixed + full * (each * groups + store);
    if (rem > 0) t += groups * (lone + (each - lone) * rem * std::sqrt(rem)) + store * rem;
    return t;
}
inline double large_us(int64_t batch, int64_t M, int64_t N, int64_t groups, int splits) {
    return tile_us((M + 255) / 256 * ((N + 255) / 256) * batch * splits,
                   static_cast<double>((groups + splits - 1) / splits), 256, 5.0, 3.5, 2.6, 10.8);
}
inline double medium_us(int64_t batch, int64_t M, int64_t N, int64_t groups, int splits) {
    return tile_us((M + 127) / 128 * ((N + 127) / 128) * batch * splits,
                   static_cast<double>((groups + splits - 1) / splits), 512, 4.0, 2.35, 1.05, 5.0);
}
inline Choice choose(int64_t batch, int64_t M, int64_t N, int64_t K, int most_splits) {
    const double dm = static_cast<double>(M), dn = static_cast<double>(N), db = static_cast<double>(batch);
    const double shares = std::ceil(dm / 32) * std::ceil(dn / 32) * db / 256;
    const double each = 1.0 + std::min(1.0, shares) * (0.6 + 0.8 * std::min(dm, 32.0) / 32);
    Choice best{kRows, 1};
    double t = 3.0 + std::max(1.0, (shares + std::ceil(shares)) / 2) *
                         std::max(0.5, each * static_cast<double>(K) / 2048);
    // tiles are counted in 32 bits on the device
    if (((dm + 127) / 128) * ((dn + 127) / 128) * db > 1e6 * 1024) return best;
    const int64_t groups = (blocks_of(K) + 15) / 16;
    for (int want = 1; want <= most_splits && want * 4 <= groups + 3; want *= 2) {
        const int s = slices_used(groups, want);
        const double sum = sum_slices_us(db, dm, dn, s);
        const double l = large_us(batch, M, N, groups, s) + sum, m = medium_us(batch, M, N, groups, s) + sum;
        if (l < t) t = l, best = {kLarge, s};
        if (m < t) t = m, best = {kMedium, s};
    }
    return best;
}

// Whether the rows of a tile, `ld` bytes apart in codes and scales and `ldc`
// floats in C, fit 32-bit offsets.
inline bool reaches(int64_t ld, int64_t ldc) {
    constexpr int64_t kReach = int64_t{1} << 31;
    return ld < kReach / 512 && ldc * 4 < kReach / 512;
}

}  // namespace product_choice

// ---- C = A op(W), A in FP32 ----
namespace weight_choice {

// W read straight into registers, 16 rows of A at a time: columns of a
// workgroup (16 nt) and slices of K, by the least predicted time.  A step of a
// workgroup's wavefronts (128 k with W transposed, 32 k as stored) takes, in
// microseconds measured on MI355X with up to 256 workgroups, for r rows of A:
//
//   16 columns 0.75 + 0.065 r   32 1.4 + 0.065 r   64 2.0 + 0.065 r   as stored, 128: 1.45
//
// and with more of them 1.2 times their share of that.
// So 16 rows x 14336 x 4096 takes 64 columns (18.8 us, against 26 with 32 and
// 40 with 16), 4 rows x 4096 x 4096 16 (8.6, against 10.3 and 14.2), 16 rows x
// 4096 x 14336 64 in 4 slices (21, against 37 with 16 unsliced), 16 x 512 x
// 8192 16 in 8 (9.9, against 20.6); as stored 16 x 4096 x 4096 takes 8 slices
// (9 and 3 for their sum, against 26.8 unsliced).
struct Direct {
    int nt, splits;
    double us;
};
inline Direct direct(bool bt, double batch, double M, double N, int64_t K, bool slices) {
    const int64_t steps = bt ? (blocks_of(K) + 3) / 4 : blocks_of(K);
    const double rows = std::ceil(M / 16) * batch, r = std::min(M, 16.0);
    Direct best{0, 1, 0};
    for (int nt = bt ? 4 : 8; nt >= (bt ? 1 : 8); nt /= 2) {
        const double tiles = rows * std::ceil(N / (16 * nt));
        const double step = !bt ? 1.45 : (nt == 4 ? 2.0 : nt == 2 ? 1.4 : 0.75) + 0.065 * r;
        for (int want = 1; want == 1 || (slices && want <= 256 && want * 8 <= steps + 7); want *= 2) {
            const int s = slices_used(steps, want);
            const double n = static_cast<double>(steps) / (8.0 * s);
            double us = 4.5 + step * std::max(std::ceil(n), 0.6 * (n + std::ceil(n)) * tiles * s / 256);
            if (s > 1) us += 1.5 + sum_slices_us(batch, M, N, s);
            if (best.nt == 0 || us < best.us) best = {nt, s, us};
        }
    }
    return best;
}

// Which kernel a product takes, and how many slices of K: the least predicted
// time, for tiles from microseconds per 32 k measured on MI355X for a lone
// tile and for a full chip (W transposed / as stored), after 4.5 that every
// launch takes and 3 that slices lose to their unequal ends:
//
//   128 x 256  two a CU     0.95 / 1.24 lone   2.19 / 2.31 full
//    64 x 256  two a CU     0.58 / 0.82 lone   1.24 / 1.34 full
//    64 x 128  three a CU   0.45 / 0.69 lone   1.07 / 1.27 full
//
// (The rates are those of K % 4 == 0: with word loads of A the first tile
// leaves room for one workgroup a CU, W transposed, which the prediction does
// not know.  Storing C has no term of its own.)
//
// 4096 x 4096 x 14336 takes the first (982 us, 1065 on a slower card, against
// 1109 and 1272), 512 x 4096 x 4096 the second in 4 slices (55 us, against 61 in
// 2, 87 unsliced and 70 with the last unsliced), 37 x 14336 x 4096 the second in
// 8 (26 us and 5 for their sum, the same in 4, against 82 unsliced).  Up to 16 rows W is always read straight
// into registers, and beyond where that is quicker: 32 x 4096 x 4096 (14.3 us
// against 17.4 with tiles, as stored 15.4 against 21.8) and 48 x 1000 x 2000
// (7.0 against 12.0), but not 48 x 14336 x 4096 (48 against 34).
constexpr int kDirect = -1;
struct Choice {
    int tile;  // 0, 1, 2 as above, or kDirect
    int splits, nt;
};
inline Choice choose(bool bt, int64_t batch, int64_t M, int64_t N, int64_t K, int most_splits) {
    struct Candidate {
        int bm, bn, slots;
        double lone[2], full[2];
    };
    static constexpr Candidate kTiles[] = {{128, 256, 512, {1.24, 0.95}, {2.31, 2.19}},
                                           {64, 256, 512, {0.82, 0.58}, {1.34, 1.24}},
                                           {64, 128, 768, {0.69, 0.45}, {1.27, 1.07}}};
    if (bt && M <= 2) return {kDirect, 1, 0};  // a kernel of their own
    const double db = static_cast<double>(batch), dm = static_cast<double>(M), dn = static_cast<double>(N);
    const Direct d = direct(bt, db, dm, dn, K, most_splits > 1);
    Choice best{kDirect, d.splits, d.nt};
    if (M <= 16) return best;
    double t = d.us;
    const int64_t chunks = (blocks_of(K) + 3) / 4;
    for (int want = 1; want <= most_splits && (want == 1 || want * 2 <= chunks); want *= 2) {
        const int s = slices_used(chunks, want);
        const double len = 4.0 * static_cast<double>((chunks + s - 1) / s);
        for (int i = 0; i < 3; ++i) {
            const Candidate &c = kTiles[i];
            const double tiles = std::ceil(dm / c.bm) * std::ceil(dn / c.bn) * db * s;
            const double full = std::floor(tiles / c.slots), rem = tiles / c.slots - full;
            double u = 4.5 + full * len * c.full[bt] +
                       (rem > 0 ? len * (c.lone[bt] + (c.full[bt] - c.lone[bt]) * rem * std::sqrt(rem)) : 0.0);
            if (s > 1) u += 3.0 + sum_slices_us(db, dm, dn, s);
            if (u < t) t = u, best = {i, s, 0};
        }
    }
    return best;
}

// Whether the tiles can run a product: a tile's rows (K rows of W as stored)
// `ldx` floats apart in A, `ldw` bytes in W and `ldc` floats in C fit 32-bit
// offsets, and a launch's lanes 2^32.
inline bool tiles_fit(bool bt, int64_t batch, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw,
                      int64_t ldc) {
    constexpr int64_t kReach = int64_t{1} << 31, kRowsM = 128, kRowsN = 256;
    const int64_t wrows = bt ? kRowsN : K;
    const double tiles = static_cast<double>((M + 63) / 64) * static_cast<double>((N + 127) / 128) *
                         static_cast<double>(batch);
    // (a stride may be near 2^60: it is divided into, never multiplied)
    return ldx < kReach / 4 / kRowsM && ldc < kReach / 4 / kRowsM && ldw < kReach / wrows && K < kReach / 8 &&
           N < kReach / 8 && tiles <= 1e6;
}

}  // namespace weight_choice

}  // namespace mx
}  // namespace gemm_f32_impl
