// The tiled product's kernels for bfloat16 operands copied to LDS directly.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_bf16(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 256) return launch_tiles_of<bf16, 256, 256, 2, 4, true>(a, g, s);
    if (g.bm == 128) return launch_tiles_of<bf16, 128, 128, 2, 2, true>(a, g, s);
    return launch_tiles_of<bf16, 64, 64, 2, 2, true>(a, g, s);
}

}  // namespace ssd
