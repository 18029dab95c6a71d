// The fused tile kernel, A stored M x K, B stored N x K.
#include "fused_tile.h"

namespace gemm_f32_impl {
namespace fused {
hipError_t launch_tile_nt(const Product &p, int tile, hipStream_t stream) {
    return launch_tile<false, true>(p, tile, stream);
}
}  // namespace fused
}  // namespace gemm_f32_impl
