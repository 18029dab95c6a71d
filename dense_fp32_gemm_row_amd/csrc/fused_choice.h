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

constexpr int kStage = 16;         // k a stage
constexpr int kMostSplits = 64;

struct Choice {
    int tile;    // index of kTiles
    int splits;  // slices of K
};

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Choice choose(int64_t batch, int64_t M, int64_t N, int64_t K, int most_splits) {
    for (int t = 0; t < kTileCount - 1; ++t)
        if (batch * div_up(M, kTiles[t].m) * div_up(N, kTiles[t].n) >= 192) return {t, 1};
    const int t = kTileCount - 1;
    const int64_t tiles = batch * div_up(M, kTiles[t].m) * div_up(N, kTiles[t].n);
    int64_t splits = std::min<int64_t>(most_splits, std::max<int64_t>(1, std::min(512 / tiles, K / 128)));
    return {t, static_cast<int>(splits)};
}

}  // namespace fused
}  // namespace gemm_f32_impl
