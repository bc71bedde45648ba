// The tiled product's kernels for float32 operands copied to LDS directly.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_f32(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 128) return launch_tiles_of<float, 128, 128, 2, 2, true>(a, g, s);
    return launch_tiles_of<float, 64, 64, 2, 2, true>(a, g, s);
}

}  // namespace ssd
