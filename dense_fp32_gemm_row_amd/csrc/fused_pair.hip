// Two independent products in one launch, in tiles of one size: the two of a layer's or
// a loss's gradient, neither of which has tiles enough to fill the GPU.
#include "fused_tile.h"

namespace gemm_f32_impl {
namespace fused {
namespace {

template <int FM, bool TA, bool TB, bool TC, bool TD>
__global__ __launch_bounds__(256, per_cu(FM)) void tile_pair_kernel(Product p, TileGrid g, Product q, TileGrid h) {
    __shared__ Room<2, 2, FM> room;
    // The tiles with more to sum come first, and every XCD takes of both: all of
    // 160 x 11731 x 1373 on two XCDs took 234 us with 1373 x 11731 x 160, this 102.
    const unsigned block = blockIdx.x, mine = static_cast<unsigned>(g.tiles), other = static_cast<unsigned>(h.tiles);
    const bool p_first = g.len >= h.len, first = block < (p_first ? mine : other);
    const unsigned at = first ? block : block - (p_first ? mine : other);
    if (first == p_first)
        one_tile<2, 2, FM, TA, TB>(p, g.tiles_m, g.tiles_n, xcd_remap(at, mine), g.len, room);
    else
        one_tile<2, 2, FM, TC, TD>(q, h.tiles_m, h.tiles_n, xcd_remap(at, other), h.len, room);
}

template <int FM>
bool launch_pair(const Product &p, const Product &q, hipStream_t stream, hipError_t *err) {
    const TileGrid g = tile_grid<2, 2, FM>(p), h = tile_grid<2, 2, FM>(q);
    if (g.tiles + h.tiles > 1 << 20) return false;
    const unsigned grid = static_cast<unsigned>(g.tiles + h.tiles);
    if (p.tb)
        tile_pair_kernel<FM, false, true, true, false><<<grid, 256, 0, stream>>>(p, g, q, h);
    else
        tile_pair_kernel<FM, false, false, true, false><<<grid, 256, 0, stream>>>(p, g, q, h);
    *err = hipGetLastError();
    return true;
}

}  // namespace

bool launch_tile_pair(const Product &p, const Product &q, int tile, hipStream_t stream, hipError_t *err) {
    return tile == 1 ? launch_pair<2>(p, q, stream, err) : launch_pair<1>(p, q, stream, err);
}

}  // namespace fused
}  // namespace gemm_f32_impl
