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
constexpr int kTileCount = 3;
constexpr int kRows = 3;           // the kernel for few rows
constexpr int kRowsMost = 32;

constexpr int kStage = 16;         // k a stage
constexpr int kMostSplits = 64;

struct Choice {
    int tile;    // index of kTiles, or kRows
    int splits;  // slices of K
    bool half;   // two fp16 parts of each value where the operands' ranges allow it
    // kRows: columns of a tile, in 16; 0: the kernel for up to 4 rows, B stored N x K
    int shape;
};

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `space`: whether there is a workspace.  `slice`: whether the sums may be slices of
// K (a row's statistics need whole ones).
// `tb`: B is stored N x K.
inline Choice choose(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, bool space, bool slice) {
    // (as stored, a lane reads 2 neighbours)
    if (M <= kRowsMost && (tb || N >= 2)) {
        const int shape = tb ? (M <= 4 ? 0 : N >= 8192 ? 4 : 1) : N >= 2048 ? 2 : 1;
        const int64_t tiles = batch * div_up(N, 16 * std::max(shape, 1));
        const int64_t splits = std::min<int64_t>(kMostSplits, std::max<int64_t>(1, std::min(256 / tiles, K / 1024)));
        return {kRows, space && slice ? static_cast<int>(splits) : 1, false, shape};
    }
    for (int t = 0; t < kTileCount - 1; ++t)
        if (batch * div_up(M, kTiles[t].m) * div_up(N, kTiles[t].n) >= 192) return {t, 1, space && K >= 64, 0};
    const int t = kTileCount - 1;
    const int64_t tiles = batch * div_up(M, kTiles[t].m) * div_up(N, kTiles[t].n);
    const int64_t splits = std::min<int64_t>(kMostSplits, std::max<int64_t>(1, std::min(512 / tiles, K / 128)));
    return {t, space && slice ? static_cast<int>(splits) : 1, false, 0};
}

// Columns of a row's piece of the cross entropy's statistics.
inline int group_columns(int64_t M) { return M <= kRowsMost ? 16 : 64; }

// Blocks of k in which the statistics of `rows` rows are taken: enough of them to fill the GPU.
inline int stat_blocks(int64_t rows, int64_t K, bool k_contiguous) {
    const int64_t units = k_contiguous ? div_up(rows, 4) : div_up(rows, 256);
    return static_cast<int>(std::max<int64_t>(1, std::min({int64_t{16}, div_up(2048, units), K / 256})));
}

}  // namespace fused
}  // namespace gemm_f32_impl
