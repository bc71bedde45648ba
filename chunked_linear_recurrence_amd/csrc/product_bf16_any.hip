// The tiled product's kernels for bfloat16 operands at any address, by way of registers.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_bf16_any(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 128) return launch_tiles_of<bf16, 128, 128, 2, 2, false>(a, g, s);
    return launch_tiles_of<bf16, 64, 64, 2, 2, false>(a, g, s);
}

}  // namespace ssd
