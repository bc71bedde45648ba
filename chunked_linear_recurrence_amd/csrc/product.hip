// Which tiled kernel takes a product, and the joining of a product whose K was split.
#include <initializer_list>

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

// A shape of tile: its size, the workgroups that a CU holds, and what they take (us): a step of K of
// one alone on its CU, of each of several that share it, and the rest of a workgroup.
struct Shape {
    int size, each_cu;
    float alone, step, fixed;
    int slots() const { return 256 * each_cu; }
};

constexpr int kMostSplits = 16, kSplitSteps = 4;        // of a tile; steps of a split at least

// Tiles of a shape for this product; those that fill the last round of workgroups only in part are
// split so that they fill it.
static ProductGrid cut(const ProductArgs &a, const Shape &sh, int64_t splits) {
    const int64_t ks = 128 / elem(a), cols = a.kind == kGated ? sh.size / 2 : sh.size, steps = (a.K + ks - 1) / ks;
    ProductGrid g;
    g.bm = g.bn = sh.size;
    g.tiles_m = (int)((a.M + sh.size - 1) / sh.size);
    g.tiles_n = (int)((a.N + cols - 1) / cols);
    const int64_t tiles = (int64_t)g.tiles_m * g.tiles_n;
    const int64_t per = (steps + splits - 1) / splits;
    g.splits = (int)((steps + per - 1) / per);
    g.steps = (int)per;
    g.rest = g.splits > 1 ? (int)(tiles % sh.slots()) : 0;
    g.full = (int)(tiles - g.rest);
    if (g.rest == 0) g.splits = 1;
    return g;
}

static int64_t part_floats(const ProductGrid &g) { return (int64_t)g.rest * g.splits * g.bm * g.bn; }

static float cost_of(const ProductArgs &a, const Shape &sh, const ProductGrid &g) {
    const int64_t ks = 128 / elem(a), steps = (a.K + ks - 1) / ks;
    auto time = [&](int64_t n, int64_t steps) {
        const int64_t rounds = n / sh.slots(), last = (n % sh.slots() + 255) / 256;      // workgroups a CU in the last
        float t = rounds * (steps * sh.each_cu * sh.step + sh.fixed);
        if (last) t += steps * (last * sh.step > sh.alone ? last * sh.step : sh.alone) + sh.fixed;
        return t;
    };
    float t = time(g.full, steps);
    if (g.rest) t += time((int64_t)g.rest * g.splits, g.steps) + 4.f + part_floats(g) * 2e-6f;
    return t;
}

// The cheapest way to cut a product, by its sizes and type alone.
static ProductGrid grid_of(const ProductArgs &a, bool dma) {
    static const Shape bf16_shapes[] = {{64, 4, 0.30f, 0.22f, 3.f}, {128, 2, 0.58f, 0.60f, 4.f}, {256, 1, 1.7f, 1.7f, 6.f}};
    static const Shape f32_shapes[] = {{64, 4, 0.5f, 0.5f, 3.f}, {128, 2, 1.9f, 1.9f, 4.f}};
    const Shape *shapes = a.dtype == 1 ? bf16_shapes : f32_shapes;
    const int n = a.dtype == 1 ? (dma ? 3 : 2) : 2;
    const int64_t ks = 128 / elem(a), steps = (a.K + ks - 1) / ks;
    ProductGrid best = cut(a, shapes[n - 1], 1);
    float least = cost_of(a, shapes[n - 1], best);
    for (int i = 0; i < n; ++i) {
        // whole, split until the last round is full, and half as far
        const ProductGrid whole = cut(a, shapes[i], 1);
        const int rest = (whole.full + whole.rest) % shapes[i].slots();
        int64_t most = rest ? shapes[i].slots() / rest : 1;
        if (most > kMostSplits) most = kMostSplits;
        if (most > steps / kSplitSteps) most = steps / kSplitSteps;
        for (int64_t splits : {(int64_t)1, (most + 1) / 2, most}) {
            if (splits < 1) continue;
            const ProductGrid g = cut(a, shapes[i], splits);
            const float t = cost_of(a, shapes[i], g);
            if (t < least) {
                least = t;
                best = g;
            }
        }
    }
    return best;
}

bool product_fits(const ProductArgs &a) {
    const int64_t cols = a.kind == kGated ? 32 : 64;
    return (a.M + 63) / 64 <= INT32_MAX / 256 / ((a.N + cols - 1) / cols);
}

size_t product_workspace_bytes(const ProductArgs &a) {
    if (product_few_rows(a)) return 0;
    const int64_t x = part_floats(grid_of(a, true)), y = part_floats(grid_of(a, false));
    return (size_t)(x > y ? x : y) * 4;
}

// Adds the partial results of shared tiles in their order and finishes them, V columns a thread.
template <typename T, ProductKind KIND>
__global__ __launch_bounds__(256) void product_join_kernel(const float *part, ProductGrid g, Epilogue ep) {
    constexpr int V = product_vec<T>();
    const int bm = g.bm, bn = g.bn, cols = KIND == kGated ? bn / 2 : bn;
    const int in = blockIdx.x * 256 + threadIdx.x, row = in / (cols / V), col = in % (cols / V) * V;
    const int id = g.full + blockIdx.y;
    const TileAt tile = tile_at(id, g);
    const int64_t m = (int64_t)tile.m * bm + row, n = (int64_t)tile.n * cols + col;
    if (row >= bm || m >= ep.M || n >= ep.N) return;
    auto sum = [&](const float *p, float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        for (int s = 0; s < g.splits; ++s, p += bm * bn)
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const f32x4 q = *reinterpret_cast<const f32x4 *>(p + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i + j] += q[j];
            }
    };
    const float *p = part + (int64_t)blockIdx.y * g.splits * bm * bn + row * bn + col;
    float v[V];
    sum(p, v);
    if constexpr (KIND == kGated) {
        float u[V];
        sum(p + bn / 2, u);
        finish_gated<T, V>(ep, m, n, v, u);
    } else {
        finish_linear<T, V>(ep, m, n, v);
    }
}

template <typename T>
static hipError_t join(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    constexpr int V = product_vec<T>();
    const int chunks = g.bm * (a.kind == kGated ? g.bn / 2 : g.bn) / V;
    const dim3 grid((uint32_t)((chunks + 255) / 256), (uint32_t)g.rest);
    if (a.kind == kGated) product_join_kernel<T, kGated><<<grid, 256, 0, s>>>(a.part, g, epilogue_of(a));
    else product_join_kernel<T, kLinear><<<grid, 256, 0, s>>>(a.part, g, epilogue_of(a));
    return hipGetLastError();
}

hipError_t launch_product(const ProductArgs &a0, hipStream_t s) {
    if (product_few_rows(a0)) return launch_product_rows(a0, s);
    ProductArgs a = a0;
    if (a.K == 1) {
        if (a.a_rows) a.a.ld = a.M;
        if (a.b_rows) a.b.ld = a.N;
    }
    const int64_t e = elem(a), ks = 128 / e;
    const int64_t brows = a.kind == kGated ? 2 * a.N : a.N, bspan = a.kind == kGated ? a.N + 256 : 256;
    const bool dma = direct(a.a, a.a_rows, a.M, a.K, a.a_rows ? ks : 256, e) &&
                     direct(a.b, a.b_rows, brows, a.K, a.b_rows ? ks : bspan, e);
    const ProductGrid g = grid_of(a, dma);
    hipError_t r;
    if (a.dtype == 1) r = dma ? launch_tiles_bf16(a, g, s) : launch_tiles_bf16_any(a, g, s);
    else r = dma ? launch_tiles_f32(a, g, s) : launch_tiles_f32_any(a, g, s);
    if (r != hipSuccess || g.rest == 0) return r;
    return a.dtype == 1 ? join<bf16>(a, g, s) : join<float>(a, g, s);
}

}  // namespace ssd
