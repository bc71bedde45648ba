// The tiled product's kernels for float32 operands copied to LDS directly.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_f32(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 128) return launch_tiles_of<float, 128, 128, 2, 2, true>(a, g, s);
    return launch_tiles_of<float, 64, 64, 2, 2, true>(a, g, s);
}

hipError_t launch_pair_f32(const ProductArgs &x, const ProductGrid &gx, const ProductArgs &w, const ProductGrid &gw,
                          bool x_first, hipStream_t s) {
    return launch_pair_of<float>(x, gx, w, gw, x_first, s);
}

}  // namespace ssd
