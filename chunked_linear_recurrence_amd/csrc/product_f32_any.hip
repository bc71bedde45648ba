// The tiled product's kernels for float32 operands at any address, by way of registers.
#include "product_tile.h"

namespace ssd {

hipError_t launch_tiles_f32_any(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (g.bm == 128) return launch_tiles_of<float, 128, 128, 2, 2, false>(a, g, s);
    return launch_tiles_of<float, 64, 64, 2, 2, false>(a, g, s);
}

}  // namespace ssd
