// Which tiled kernel takes a product, and the joining of a product whose K was split.
#include "product.h"

namespace ssd {

static int64_t elem(const ProductArgs &a) { return a.dtype == 1 ? 2 : 4; }

// Whether an operand's 16-byte pieces all lie on 16 bytes and inside a row, with the tile's
// offsets below 2^31: `span` rows of a tile where k is contiguous, of k otherwise.
static bool direct(const Operand &o, bool rows_contiguous, int64_t rows, int64_t k, int64_t span, int64_t e) {
    const int64_t along = rows_contiguous ? rows : k, across = rows_contiguous ? k : rows;
    if ((uintptr_t)o.p & 15u || along * e % 16 != 0) return false;
    if (across > 1 && o.ld * e % 16 != 0) return false;
    if (rows_contiguous && o.ld < rows) return false;     // lines past K have to lie past the last one
    return o.ld <= (int64_t)0x70000000 / e / span;
}

// Tiles of BM x BN and the steps of each split for a product of `splits` splits
static ProductGrid cut(const ProductArgs &a, int64_t bm, int64_t bn, int64_t splits) {
    const int64_t ks = 128 / elem(a), cols = a.kind == kGated ? bn / 2 : bn, steps = (a.K + ks - 1) / ks;
    const int64_t per = (steps + splits - 1) / splits;
    return {(int)((a.M + bm - 1) / bm), (int)((a.N + cols - 1) / cols), (int)((steps + per - 1) / per), (int)per};
}
static int64_t tiles_of(const ProductGrid &g) { return (int64_t)g.tiles_m * g.tiles_n; }

static ProductGrid grid_of(const ProductArgs &a) {
    const ProductGrid g = cut(a, 128, 128, 1);
    const int64_t tiles = tiles_of(g);
    if (tiles >= 192) return g;
    int64_t splits = 512 / tiles;
    if (splits > g.steps / 4) splits = g.steps / 4;
    return cut(a, 128, 128, splits < 1 ? 1 : splits);
}

static bool big_tiles(const ProductArgs &a, ProductGrid *g) {
    if (a.dtype != 1) return false;
    *g = cut(a, 256, 256, 1);
    const int64_t big = (tiles_of(*g) + 255) / 256, small = (tiles_of(cut(a, 128, 128, 1)) + 511) / 512;
    return 8 * big <= 5 * small;
}

bool product_fits(const ProductArgs &a) {
    return grid_fits(tiles_of(grid_of(a)), 256);
}

size_t product_workspace_bytes(const ProductArgs &a) {
    const ProductGrid g = grid_of(a);
    return g.splits > 1 ? (size_t)g.splits * a.M * a.N * (a.kind == kGated ? 2 : 1) * 4 : 0;
}

// Adds the splits' sums in their order and finishes the results, V columns a thread.
template <typename T, ProductKind KIND>
__global__ __launch_bounds__(256) void product_join_kernel(const float *part, int splits, Epilogue ep) {
    constexpr int V = product_vec<T>();
    const int64_t chunks = (ep.N + V - 1) / V, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= ep.M * chunks) return;
    const int64_t m = id / chunks, n = id % chunks * V, cols = KIND == kGated ? 2 * ep.N : ep.N;
    const int left = (int)min(ep.N - n, (int64_t)V);
    const bool whole = left == V && ep.N % 4 == 0;
    auto sum = [&](const float *p, float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        for (int s = 0; s < splits; ++s, p += ep.M * cols) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float q[4];
                load_some<float, 4>(p + i, left - i, whole, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i + j] += q[j];
            }
        }
    };
    const float *p = part + m * cols + n;
    float v[V];
    sum(p, v);
    if constexpr (KIND == kGated) {
        float u[V];
        sum(p + ep.N, u);
        finish_gated<T, V>(ep, m, n, v, u);
    } else {
        finish_linear<T, V>(ep, m, n, v);
    }
}

template <typename T>
static hipError_t join(const ProductArgs &a, int splits, hipStream_t s) {
    constexpr int V = product_vec<T>();
    const uint32_t blocks = (uint32_t)((a.M * ((a.N + V - 1) / V) + 255) / 256);
    if (a.kind == kGated) product_join_kernel<T, kGated><<<blocks, 256, 0, s>>>(a.part, splits, epilogue_of(a));
    else product_join_kernel<T, kLinear><<<blocks, 256, 0, s>>>(a.part, splits, epilogue_of(a));
    return hipGetLastError();
}

hipError_t launch_product(const ProductArgs &a0, hipStream_t s) {
    ProductArgs a = a0;
    if (a.K == 1) {
        if (a.a_rows) a.a.ld = a.M;
        if (a.b_rows) a.b.ld = a.N;
    }
    const int64_t e = elem(a), ks = 128 / e;
    const int64_t brows = a.kind == kGated ? 2 * a.N : a.N, bspan = a.kind == kGated ? a.N + 256 : 256;
    const bool dma = direct(a.a, a.a_rows, a.M, a.K, a.a_rows ? ks : 256, e) &&
                     direct(a.b, a.b_rows, brows, a.K, a.b_rows ? ks : bspan, e);
    ProductGrid g;
    if (dma && big_tiles(a, &g)) return launch_tiles_bf16_big(a, g, s);
    g = grid_of(a);
    hipError_t r;
    if (a.dtype == 1) r = dma ? launch_tiles_bf16(a, g, s) : launch_tiles_bf16_any(a, g, s);
    else r = dma ? launch_tiles_f32(a, g, s) : launch_tiles_f32_any(a, g, s);
    if (r != hipSuccess || g.splits == 1) return r;
    return a.dtype == 1 ? join<bf16>(a, g.splits, s) : join<float>(a, g.splits, s);
}

}  // namespace ssd
