// The tiled product's kernels for bfloat16 operands copied to LDS directly.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_bf16(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    return launch_tiles_of<bf16, 128, 128, 2, 2, true>(a, g, s);
}

}  // namespace ssd
