// Which kernel a fused product takes, from its sizes alone (host code,
// also compiled by a CPU test).
#pragma once

#include <algorithm>
#include <cstdint>

namespace gemm_f32_impl {
namespace fused {

struct TileSize {
    int m, n;
};
constexpr TileSize kTiles[] = {{256, 256}, {128, 128}, {64, 128}};
constexpr int kRows = 3;           // the kernel for few rows and small products
constexpr int kRowsMost = 32;      // rows for which it, and only it, is taken
// Tokens for which the cross entropy's statistics are kept by 16 columns, not 64:
// the kernel for small products holds fewer than 64.
constexpr int kFineTokens = 512;

constexpr int kStage = 16;         // k a stage
constexpr int kMostSplits = 32;

struct Choice {
    int tile;    // index of kTiles, or kRows
    int splits;  // slices of K
    bool half;   // two fp16 parts of each value where the operands' ranges allow it
    // kRows: rows and columns of a tile in 16, 16 r + c (c <= N where B is stored K x
    // N, r <= M where A is stored K x M); 0: the kernel for up to 4 rows, B stored N x K
    int shape;
};

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a kernel's tile takes, in nanoseconds: `lone` a k and `fixed` besides where a
// CU has one of them, `shared` a k and `each` besides of every one where it has more.
// Fitted to 5600 times of 270 products of 33 to 8192 rows (three operand forms, 90 sizes
// drawn evenly over their logarithms): the choice is 2.2% off the best of all
// kernels and slices on average.
struct Rate {
    Choice kind;
    int m, n;
    double lone, fixed, shared, each;
};
constexpr Rate kRates[] = {
    {{kRows, 1, false, 17}, 16, 16, 2.6, 884, 2.8, 670},     {{kRows, 1, false, 18}, 16, 32, 4.2, 1040, 4.1, 1079},
    {{kRows, 1, false, 34}, 32, 32, 6.6, 2167, 6.9, 1765},   {{kRows, 1, false, 36}, 32, 64, 11.5, 2310, 11.5, 2447},
    {{kRows, 1, false, 66}, 64, 32, 11.5, 2221, 11.3, 2868}, {{2, 1, false, 0}, 64, 128, 29.2, 5210, 23.3, 3423},
    {{1, 1, false, 0}, 128, 128, 33.0, 9106, 36.0, 5713},    {{1, 1, true, 0}, 128, 128, 25.0, 2473, 22.5, 4970},
    {{0, 1, false, 0}, 256, 256, 96.6, 33397, 129.1, 25567}, {{0, 1, true, 0}, 256, 256, 50.8, 29554, 73.5, 30865},
};
constexpr double kCus = 256;
constexpr double kBytesNs = 5500;                           // memory, reading
constexpr double kSumNs = 2660, kSumBytesNs = 5700;         // adding slices
constexpr double kStatsNs = 8870, kStatsBytesNs = 8120;     // looking at the rows' ranges

inline double predicted(const Rate &r, int64_t batch, int64_t M, int64_t N, int64_t K, int64_t splits) {
    const double tiles = static_cast<double>(batch) * div_up(M, r.m) * div_up(N, r.n) * splits / kCus;
    const double k = static_cast<double>(div_up(K, splits)), alone = r.lone * k + r.fixed;
    const double turns = tiles <= 6 ? static_cast<double>(static_cast<int64_t>(tiles + 0.999999)) : tiles + 0.5;
    double t = tiles > 1 ? std::max(alone, turns * (r.shared * k + r.each)) : alone;
    const double mk = static_cast<double>(M) * K, nk = static_cast<double>(N) * K, mn = static_cast<double>(M) * N;
    t = std::max(t, 4 * batch * (mk + nk + mn) / kBytesNs);
    if (splits > 1) t += kSumNs + 4 * batch * (splits + 1) * mn / kSumBytesNs;
    if (r.kind.half) t += kStatsNs + 4 * batch * (mk + nk) / kStatsBytesNs;
    return t;
}

// What the product is for: statistics of whole rows allow no slices, and of many
// tokens only the tiles; of the loss's probabilities, whose small values may be all that
// counts in a gradient, next to no two fp16 parts hold enough (a word's probability of
// 2^-17 beside its target's 1 leaves them 2^-22 of it), so they take three bf16 parts.
enum Use { kPlain, kStatistics, kProbabilities };

// `tb`: B is stored N x K.  `space`: whether there is a workspace.
inline Choice choose(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, bool space, Use use) {
    const bool slice = space && use != kStatistics;
    // Few rows: reading B is the work, in tiles as wide as leaves enough of them (as
    // stored, a lane reads 2 neighbours): 16 x 14336 x 4096, B transposed, 47 us with 64
    // columns and 65 with 16, 16 x 4096 x 4096 43 and 18; 5 x 1792 x 78080, B as stored,
    // 119 us with 32 columns in 4 slices of K, 314 with 16 in one.
    if (M <= kRowsMost) {
        const int c = tb ? (N >= 8192 && M > 4 ? 4 : 1) : N >= 1024 ? 2 : 1;
        const int shape = tb && M <= 4 ? 0 : (M <= 16 ? 16 : 32) + c;
        const int64_t tiles = batch * div_up(N, 16 * c), most = (tb ? 256 : 512) / tiles;
        const int64_t splits = std::min<int64_t>(kMostSplits, std::max<int64_t>(1, std::min(most, K / 1024)));
        return {kRows, slice ? static_cast<int>(splits) : 1, false, shape};
    }
    // Up to 3 columns of a B stored K x N: a tile's loads take 4 neighbours, so none serves
    // (8192 x 1 x 4096 26 us, by a tile's loop for any shape 244).  Statistics are of a B
    // stored N x K.
    const bool few = !tb && N < 4 && use != kStatistics;
    Choice best{};
    double least = 0;
    for (const Rate &r : kRates) {
        if (r.kind.half && (!space || use == kProbabilities || K < 64 || K > (int64_t{1} << 22))) continue;
        if (r.kind.tile == kRows ? (use == kStatistics && M > kFineTokens) || (!tb && (r.kind.shape & 15) > N) : few) continue;
        const int64_t tiles = batch * div_up(M, r.m) * div_up(N, r.n);
        for (int64_t splits = 1; splits <= (slice ? kMostSplits : 1); splits *= 2) {
            if (splits > 1 && (tiles * splits > 2048 || K < 64 * splits)) break;
            const double t = predicted(r, batch, M, N, K, splits);
            if (least > 0 && t >= least) continue;
            least = t;
            best = r.kind;
            best.splits = static_cast<int>(splits);
        }
    }
    return best;
}

// Columns of a row's piece of the cross entropy's statistics.
inline int group_columns(int64_t tokens) { return tokens <= kFineTokens ? 16 : 64; }

// Blocks of k in which the statistics of `rows` rows are taken: enough of them to fill the GPU.
inline int stat_blocks(int64_t rows, int64_t K, bool k_contiguous) {
    const int64_t units = k_contiguous ? div_up(rows, 4) : div_up(rows, 256);
    return static_cast<int>(std::max<int64_t>(1, std::min({int64_t{k_contiguous ? 16 : 64}, div_up(1024, units), K / (k_contiguous ? 256 : 64)})));
}

}  // namespace fused
}  // namespace gemm_f32_impl
