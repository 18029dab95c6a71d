// The fused tile kernel, A stored K x M, B stored N x K.
#include "fused_tile.h"

namespace gemm_f32_impl {
namespace fused {
hipError_t launch_tile_tt(const Product &p, int tile, hipStream_t stream) {
    return launch_tile<true, true>(p, tile, stream);
}
}  // namespace fused
}  // namespace gemm_f32_impl
