// Which tiled kernel takes a product, and the joining of a product whose K was split.
#include <initializer_list>

#include "product.h"

namespace ssd {

static int64_t elem(const ProductArgs &a) { return a.dtype == 1 ? 2 : 4; }

// An operand as lines of contiguous values.
struct Lines {
    int64_t count, length, ld;
    int64_t span;                 // lines a tile's offsets reach over
    bool rows;                    // a line is one k, its values rows
};
static Lines lines_of(const ProductArgs &a, bool of_b) {
    const int64_t ks = 128 / elem(a), rows = !of_b ? a.M : a.kind == kGated ? 2 * a.N : a.N;
    const bool contiguous = of_b ? a.b_rows : a.a_rows;
    const int64_t ld = of_b ? a.b.ld : a.a.ld;
    // one line of k has no stride of its own; lines past K, at which a tile's offsets point, lie past it
    if (contiguous) return {a.K, rows, a.K == 1 && ld < rows ? rows : ld, ks, true};
    return {rows, a.K, ld, of_b && a.kind == kGated ? a.N + 256 : 256, false};
}

// Whether 16-byte pieces from the lines' starts on cover them without reaching into what lies
// behind, with a tile's offsets below 2^31, if the first line starts on 16 bytes.
static bool direct(const Lines &o, int64_t e) {
    if (o.length * e % 16 != 0) return false;
    if (o.count > 1 && o.ld * e % 16 != 0) return false;
    if (o.rows && o.count > 1 && o.ld < o.length) return false;     // lines past K have to lie past the last one
    return o.ld <= (int64_t)0x70000000 / e / o.span;
}

static int64_t packed_ld(const Lines &o, int64_t e) { return (o.length * e + 15) / 16 * (16 / e); }
static size_t packed_bytes(const Lines &o, int64_t e) { return (size_t)(o.count * packed_ld(o, e) * e + 255) / 256 * 256; }
static bool can_pack(const Lines &o, int64_t e) { return packed_ld(o, e) <= (int64_t)0x70000000 / e / o.span; }

// A shape of tile: its size, the workgroups that a CU holds, and what they take (us): a step of K of
// one alone on its CU, of each of several that share it, and the rest of a workgroup.
struct Shape {
    int size, each_cu;
    float alone, step, fixed;
    int slots() const { return 256 * each_cu; }
};

// For operands copied to LDS directly and for those from any address
constexpr Shape bf16_dma[] = {{64, 4, 0.30f, 0.22f, 3.f}, {128, 2, 0.58f, 0.60f, 4.f}, {256, 1, 1.7f, 1.7f, 6.f}};
constexpr Shape bf16_any[] = {{64, 4, 0.30f, 0.32f, 3.f}, {128, 2, 0.9f, 0.9f, 4.f}};
constexpr Shape f32_dma[] = {{64, 4, 0.5f, 0.5f, 3.f}, {128, 2, 1.9f, 1.9f, 14.f}};
constexpr Shape f32_any[] = {{64, 4, 0.7f, 0.8f, 3.f}, {128, 2, 2.5f, 2.4f, 14.f}};
constexpr int kPairTiles = 1 << 20;                     // of two products in one launch, well within a grid's range

// A split's partial results, written and read again, are to be no more than what it reads for them: 128 KB
// of a tile of 128 and 4 steps of 32 KB (of a tile of 64 a half, of 256 twice of it).  By steps of a
// split at least, 2, 4 and 8: float32 65 x 1024 x 256 11.8, 10.3 and 11.3 us, 65 x 512 x 128 9.1, 9.1 and
// 13.4, bfloat16 100 x 4096 x 64 11.5, 11.6 and 10.4.  By splits of a tile, 8, 16 and 32: bfloat16 128 x
// 16384 x 128 16.9, 15.1 and 18.0, float32 42.1, 27.2 and 24.1; 84 and 309 whole.
constexpr int kMostSplits = 16, kSplitSteps = 4;        // of a tile; steps of a split at least

// Tiles of a shape for this product; those beyond a whole number for each CU are split.
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
    g.rest = g.splits > 1 ? (int)(tiles % 256) : 0;
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
    // partial results: a launch, and their stores and the join's reads (12.6 M of them: 12 us in the join)
    if (g.rest) t += time((int64_t)g.rest * g.splits, g.steps) + 4.f + part_floats(g) * 2e-6f;
    return t;
}

// The cheapest way to cut a product, by its sizes and type alone.  Small tiles give every CU work,
// large ones read less from LDS and the caches for each product: us in tiles of 64, 128 and 256,
// bfloat16, 512 x 2048 x 2048 13.5, 23.3, 32.9; 2048 x 2048 x 4096 55.9, 40.0, 49.3; 4096^3 189, 134,
// 109; float32 512 x 1024 x 1024 16.8, 29.2 (whole tiles of 64: 21.6), 8192 x 64 x 2048 36, 67, 8192 x
// 256 x 4096 144, 175 (a tile of 128 alone stores for 14 us, twice its bytes' time: a lane's accesses of 16
// bytes lie 64 apart from its neighbours').
static ProductGrid grid_of(const ProductArgs &a, bool dma, float *cost) {
    const Shape *shapes = a.dtype == 1 ? (dma ? bf16_dma : bf16_any) : dma ? f32_dma : f32_any;
    const int n = a.dtype == 1 && dma ? 3 : 2;
    const int64_t ks = 128 / elem(a), steps = (a.K + ks - 1) / ks;
    ProductGrid best = cut(a, shapes[n - 1], 1);
    float least = cost_of(a, shapes[n - 1], best);
    for (int i = 0; i < n; ++i) {
        // whole, or the tiles that do not make a whole number for each CU split until they give each one
        // workgroup, as many as it holds, or half of that
        const ProductGrid whole = cut(a, shapes[i], 1);
        const int rest = (whole.full + whole.rest) % 256;
        const int64_t by_steps = steps / kSplitSteps, most = by_steps < 1 ? 1 : by_steps < kMostSplits ? by_steps : kMostSplits;
        const int64_t one = rest ? 256 / rest : 1, all = rest ? shapes[i].slots() / rest : 1;
        int64_t tried = 0;
        for (int64_t want : {(int64_t)1, one, (all + 1) / 2, all}) {
            const int64_t splits = want < most ? want : most;
            if (splits == tried) continue;
            tried = splits;
            const ProductGrid g = splits == 1 ? whole : cut(a, shapes[i], splits);
            const float t = cost_of(a, shapes[i], g);
            if (t < least) {
                least = t;
                best = g;
            }
        }
    }
    *cost = least;
    return best;
}

// How a product runs, by its sizes, strides and type alone.  Operands whose lines are not whole
// pieces of 16 bytes are read from any address by way of registers, or, where the product is long
// enough to win that back (6 us and 0.6 for each MB), laid out anew in the workspace first:
// 4095^3 in bfloat16 217 us by way of registers and 134 so, 1999 x 777 x 1025 in float32 63 and 45.
struct Plan {
    bool dma, pack_a, pack_b;
    ProductGrid g;
    size_t part, total;           // the partial results' place in the workspace (packed operands first), its bytes
    float cost;
};
static float packing_cost(size_t bytes) { return bytes ? 6.f + bytes * 6e-7f : 0.f; }
static size_t part_bytes(const ProductGrid &g) { return (size_t)part_floats(g) * 4; }

static Plan plan_of(const ProductArgs &a) {
    const int64_t e = elem(a);
    const Lines la = lines_of(a, false), lb = lines_of(a, true);
    Plan p = {true, !direct(la, e), !direct(lb, e), {}, 0, 0, 0.f};
    float any;
    p.g = grid_of(a, true, &p.cost);
    if (p.pack_a || p.pack_b) {
        const ProductGrid g = grid_of(a, false, &any);
        const size_t bytes = (p.pack_a ? packed_bytes(la, e) : 0) + (p.pack_b ? packed_bytes(lb, e) : 0);
        const bool can = (!p.pack_a || can_pack(la, e)) && (!p.pack_b || can_pack(lb, e));
        if (can && p.cost + packing_cost(bytes) < any) {
            p.part = bytes;
            p.cost += packing_cost(bytes);
        } else {
            p.cost = any;
            p.dma = p.pack_a = p.pack_b = false;
            p.g = g;
        }
    }
    p.total = p.part + part_bytes(p.g);
    return p;
}

bool product_fits(const ProductArgs &a) {
    const int64_t cols = a.kind == kGated ? 32 : 64;
    const int64_t down = (a.M + 63) / 64, across = (a.N + cols - 1) / cols;
    if (down > (INT64_C(1) << 30) / across) return false;       // tiles are counted in int
    if (down * across <= 1 << 22) return true;                   // whatever their shape
    float cost;
    for (bool dma : {false, true}) {
        const ProductGrid g = grid_of(a, dma, &cost);
        if (!grid_fits(g.full + (int64_t)g.rest * g.splits, g.bm == 256 ? 512 : 256)) return false;
    }
    return true;
}

// Tensors may start off 16 bytes, which their sizes do not tell: the product then runs from any
// address.
static size_t bytes_of(const ProductArgs &a, const Plan &p) {
    if (!p.dma) return p.total;
    float cost;
    const size_t any = part_bytes(grid_of(a, false, &cost));
    return p.total > any ? p.total : any;
}
size_t product_workspace_bytes(const ProductArgs &a) { return product_few_rows(a) ? 0 : bytes_of(a, plan_of(a)); }

// Lines of `length` values at ld to lines of whole pieces, the rest of the last piece zeros: up to
// three operands (blockIdx.y) in one launch, a wave for each line, four pieces of a lane on their way.
struct Packing {
    const void *src;
    int64_t ld, lines, length;
    void *dst;
};
template <typename T>
__global__ __launch_bounds__(256) void product_pack_kernel(Packing a, Packing b, Packing c) {
    constexpr int V = product_vec<T>(), U = 4;
    const Packing p = blockIdx.y == 0 ? a : blockIdx.y == 1 ? b : c;
    const int lane = threadIdx.x % 64;
    const int64_t whole = p.length / V, pieces = (p.length + V - 1) / V;
    for (int64_t line = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; line < p.lines; line += (int64_t)gridDim.x * 4) {
        const T *from = reinterpret_cast<const T *>(p.src) + line * p.ld;
        u32x4 *to = reinterpret_cast<u32x4 *>(p.dst) + line * pieces;
        for (int64_t at = lane; at < whole; at += 64 * U) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) __builtin_memcpy(&v[u], from + min(at + 64 * u, whole - 1) * V, 16);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (at + 64 * u < whole) to[at + 64 * u] = v[u];
        }
        if (lane == 0 && whole < pieces) {
            T v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = whole * V + k < p.length ? from[whole * V + k] : from_f32<T>(0.f);
            __builtin_memcpy(&to[whole], v, 16);
        }
    }
}

static hipError_t pack_launch(const Packing *job, int n, int64_t e, hipStream_t s) {
    int64_t lines = 0;
    for (int i = 0; i < n; ++i)
        if (job[i].lines > lines) lines = job[i].lines;
    const int64_t blocks = (lines + 3) / 4;
    const dim3 grid((uint32_t)(blocks < 2048 ? blocks : 2048), (uint32_t)n);
    const Packing &b = job[n > 1 ? 1 : 0], &c = job[n > 2 ? 2 : 0];
    if (e == 2) product_pack_kernel<bf16><<<grid, 256, 0, s>>>(job[0], b, c);
    else product_pack_kernel<float><<<grid, 256, 0, s>>>(job[0], b, c);
    return hipGetLastError();
}

// Lays operands anew at `to`, one behind the other.
static hipError_t pack(const Plan &p, const Lines &la, const Lines &lb, ProductArgs *a, char *to, hipStream_t s) {
    const int64_t e = elem(*a);
    Packing job[2];
    int n = 0;
    auto add = [&](const Lines &o, Operand *op) {
        job[n++] = {op->p, o.ld, o.count, o.length, to};
        op->p = to;
        op->ld = packed_ld(o, e);
        if (o.rows) op->size = op->ld;
        to += packed_bytes(o, e);
    };
    if (p.pack_a) add(la, &a->a);
    if (p.pack_b) add(lb, &a->b);
    return n ? pack_launch(job, n, e, s) : hipSuccess;
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
    const Lines la = lines_of(a, false), lb = lines_of(a, true);
    a.a.size = la.length;
    a.b.size = lb.length;
    a.a.ld = la.ld;
    a.b.ld = lb.ld;
    Plan p = plan_of(a);
    auto at16 = [](const void *q) { return ((uintptr_t)q & 15u) == 0; };
    if (p.dma && ((!p.pack_a && !at16(a.a.p)) || (!p.pack_b && !at16(a.b.p)))) {
        float cost;
        p = {false, false, false, grid_of(a, false, &cost), 0, 0, cost};
    }
    char *ws = reinterpret_cast<char *>(a.part);
    hipError_t r = pack(p, la, lb, &a, ws, s);
    if (r != hipSuccess) return r;
    a.part = reinterpret_cast<float *>(ws + p.part);
    if (a.dtype == 1) r = p.dma ? launch_tiles_bf16(a, p.g, s) : launch_tiles_bf16_any(a, p.g, s);
    else r = p.dma ? launch_tiles_f32(a, p.g, s) : launch_tiles_f32_any(a, p.g, s);
    if (r != hipSuccess || p.g.rest == 0) return r;
    return a.dtype == 1 ? join<bf16>(a, p.g, s) : join<float>(a, p.g, s);
}

// A gradient's two products in one launch, where tiles of 64 suit each and their work together loads the CUs more evenly than in turn: dpre, x and the weight laid out anew once, tiles
// whole.  Both gradients, us in turn and together: float32 1999 x 777 x 1025 98 and 80, 1024^3 45.6
// and 35.6, bfloat16 2048 x 768 x 1024 29.6 and 19.4, 3000 x 300 x 2000 54 and 33; long sums of few tiles stay split, by themselves:
// bfloat16 16384 x 128 x 256 20 and 126, 4096 x 256 x 512 17.3 and 21.3.
struct PairPlan {
    bool pair, pack_d, pack_x, pack_w;       // dpre, x and the weight are laid out anew
    ProductGrid gx, gw;
    size_t bytes;
};
static PairPlan pair_of(const ProductArgs &x, const ProductArgs &w, const Plan &by_x, const Plan &by_w) {
    PairPlan p = {};
    const Shape &sh = (x.dtype == 1 ? bf16_dma : f32_dma)[0];
    const int64_t e = elem(x), ks = 128 / e;
    if ((by_x.dma && by_x.g.bm != sh.size) || (by_w.dma && by_w.g.bm != sh.size)) return p;
    const Lines dx = lines_of(x, false), dw = lines_of(w, false), lw = lines_of(x, true), lx = lines_of(w, true);
    p.pack_d = !direct(dx, e) || !direct(dw, e);
    p.pack_w = !direct(lw, e);
    p.pack_x = !direct(lx, e);
    if ((p.pack_d && !(can_pack(dx, e) && can_pack(dw, e))) || (p.pack_w && !can_pack(lw, e)) || (p.pack_x && !can_pack(lx, e)))
        return p;
    p.bytes = (p.pack_d ? packed_bytes(dw, e) : 0) + (p.pack_w ? packed_bytes(lw, e) : 0) + (p.pack_x ? packed_bytes(lx, e) : 0);
    p.gx = cut(x, sh, 1);
    p.gw = cut(w, sh, 1);
    if ((int64_t)p.gx.full + p.gw.full > kPairTiles) return p;
    // a CU's share of both and a part of the longer tile for the uneven end, or the longer tile alone;
    // against both in turn and what lies between two launches (3 us)
    const float sx = (x.K + ks - 1) / ks, sw = (w.K + ks - 1) / ks, longer = sx > sw ? sx : sw;
    const float each = (p.gx.full * sx + p.gw.full * sw) / 256 + 0.25f * longer;
    const float both = (each * sh.step > longer * sh.alone ? each * sh.step : longer * sh.alone) + sh.fixed;
    p.pair = both + packing_cost(p.bytes) < by_x.cost + by_w.cost + 3.f;
    return p;
}

size_t product_grads_workspace_bytes(const ProductArgs &x, const ProductArgs &w) {
    const Plan by_x = plan_of(x), by_w = plan_of(w);
    const size_t a = bytes_of(x, by_x), b = bytes_of(w, by_w);
    const PairPlan p = pair_of(x, w, by_x, by_w);
    const size_t both = p.pair ? p.bytes : 0;
    return both > a && both > b ? both : a > b ? a : b;
}

hipError_t launch_product_grads(const ProductArgs &x, const ProductArgs &w, hipStream_t s) {
    auto at16 = [](bool packed, const void *q) { return packed || ((uintptr_t)q & 15u) == 0; };
    const PairPlan p = x.y && w.y ? pair_of(x, w, plan_of(x), plan_of(w)) : PairPlan{};
    if (!p.pair || !at16(p.pack_d, x.a.p) || !at16(p.pack_w, x.b.p) || !at16(p.pack_x, w.b.p)) {
        const hipError_t r = x.y ? launch_product(x, s) : hipSuccess;
        return r == hipSuccess && w.y ? launch_product(w, s) : r;
    }
    ProductArgs ax = x, aw = w;
    const int64_t e = elem(x);
    const Lines ld = lines_of(w, false), lw = lines_of(x, true), lx = lines_of(w, true);
    aw.a.size = ld.length;
    ax.b.size = lw.length;
    aw.b.size = lx.length;
    aw.a.ld = ld.ld;
    ax.b.ld = lw.ld;
    aw.b.ld = lx.ld;
    Packing job[3];
    int n = 0;
    char *to = reinterpret_cast<char *>(x.part);
    auto add = [&](const Lines &o, Operand *op) {
        job[n++] = {op->p, o.ld, o.count, o.length, to};
        op->p = to;
        op->ld = op->size = packed_ld(o, e);
        to += packed_bytes(o, e);
    };
    if (p.pack_d) {
        add(ld, &aw.a);
        ax.a.p = aw.a.p;
        ax.a.ld = aw.a.ld;
    }
    if (p.pack_w) add(lw, &ax.b);
    if (p.pack_x) add(lx, &aw.b);
    if (n) {
        const hipError_t r = pack_launch(job, n, e, s);
        if (r != hipSuccess) return r;
    }
    const bool x_first = x.K >= w.K;                            // the longer tiles first
    return x.dtype == 1 ? launch_pair_bf16(ax, p.gx, aw, p.gw, x_first, s) : launch_pair_f32(ax, p.gx, aw, p.gw, x_first, s);
}

}  // namespace ssd
