// The tiled product's kernels for bfloat16 operands copied to LDS directly, large tiles.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_bf16_big(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    return launch_tiles_of<bf16, 256, 256, 2, 4, true>(a, g, s);
}

}  // namespace ssd
