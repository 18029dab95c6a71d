// The fused tile kernel, A stored M x K, B stored K x N.
#include "fused_tile.h"

namespace gemm_f32_impl {
namespace fused {
hipError_t launch_tile_nn(const Product &p, int tile, hipStream_t stream) {
    return launch_tile<false, false>(p, tile, stream);
}
}  // namespace fused
}  // namespace gemm_f32_impl
