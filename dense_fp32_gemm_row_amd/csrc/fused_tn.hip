// The fused tile kernel, A stored K x M, B stored K x N.
#include "fused_tile.h"

namespace gemm_f32_impl {
namespace fused {
hipError_t launch_tile_tn(const Product &p, int tile, hipStream_t stream) {
    return launch_tile<true, false>(p, tile, stream);
}
}  // namespace fused
}  // namespace gemm_f32_impl
