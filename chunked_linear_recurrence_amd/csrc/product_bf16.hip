// The tiled product's kernels for bfloat16 operands copied to LDS directly.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_bf16(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 256) return launch_tiles_of<bf16, 256, 256, 2, 4, true>(a, g, s);
    if (g.bm == 128) return launch_tiles_of<bf16, 128, 128, 2, 2, true>(a, g, s);
    return launch_tiles_of<bf16, 64, 64, 2, 2, true>(a, g, s);
}

hipError_t launch_pair_bf16(const ProductArgs &x, const ProductGrid &gx, const ProductArgs &w, const ProductGrid &gw,
                          bool x_first, hipStream_t s) {
    return launch_pair_of<bf16>(x, gx, w, gw, x_first, s);
}

}  // namespace ssd
