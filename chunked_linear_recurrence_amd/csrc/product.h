// Matrix products with what follows them in one kernel: arguments, launch functions and the
// arithmetic that their kernels share.
//
//     linear   pre = A B^T + bias;              y = act(pre) + residual
//     gated    [g | u] = A B^T + bias;          h = act(g) u         (B: F rows of g, F of u)
//     plain    c = A B^T
//
// Every sum over k is held in float32 in the matrix units' accumulators; results are rounded
// once, when they are stored.  pre, which a backward takes, is float32 or of the activations' type.
// The gradient by it is rounded to that type before its two products, whose matrix units take no
// float32 at the rate of bfloat16.  Errors in the 2-norm of the gradients of 8192 x 2048 x (2 x 5632)
// against 64 bits, in bfloat16: 0.0024 with pre in float32, 0.0030 in bfloat16 and 0.0017 by the
// last rounding alone; forward and backward 359 + 721 us and 332 + 686.
#pragma once

#include "ssd_block.h"

namespace ssd {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

enum Act { kActNone = 0, kActSilu = 1, kActGelu = 2 };

// An operand [rows, K] of a product: element (r, k) at p + r * ld + k, or, where the rows are
// the contiguous axis (the transposed operands of a backward pass), at p + k * ld + r.
struct Operand {
    const void *p;
    int64_t ld;
    int64_t size;                 // values that may be read of a line, where the rows are contiguous
};

enum ProductKind { kLinear, kGated, kPlain };

struct ProductArgs {
    int64_t M, N, K;              // c [M, N]; gated: N = F, and B has 2 F rows
    int dtype;
    ProductKind kind;
    bool a_rows, b_rows;          // the operand's rows are its contiguous axis
    Operand a, b;
    const void *bias;             // [N], gated [2 F]; act dtype, or null
    const void *residual;         // [M, N] at residual_ld, or null (linear)
    int64_t residual_ld;
    int act;
    void *y;                      // [M, N]
    void *pre;                    // linear [M, N], gated [M, 2 F]; or null
    bool pre_f32;                 // pre is float32, whatever the activations' type
    float *part;                  // workspace of tiles whose K is split: [rest, splits, bm, bn]
};

// How one launch cuts its product into tiles: `full` of them take one workgroup each, and each of
// the `rest` behind them `splits` workgroups, of `steps` steps of K (128 bytes a row) each, whose
// partial results a second kernel adds.
struct ProductGrid {
    int bm, bn;                   // rows and columns of B of a tile (gated: both halves')
    int tiles_m, tiles_n;
    int full, rest, splits, steps;
};

// Where tile `id` lies: in groups of 4 columns, row by row within a group, so that the 32 tiles that
// an XCD (own L2) holds at a time share their operands.
struct TileAt {
    int m, n;
};
__host__ __device__ inline TileAt tile_at(int id, const ProductGrid &g) {
    constexpr int G = 4;
    const int group = id / (G * g.tiles_m), first = group * G, left = g.tiles_n - first, width = left < G ? left : G;
    const int in = id - group * G * g.tiles_m;
    return {in / width, first + in % width};
}

bool product_fits(const ProductArgs &a);                  // its work is within a launch
size_t product_workspace_bytes(const ProductArgs &a);
hipError_t launch_product(const ProductArgs &a, hipStream_t s);
// A gradient's products by x (dpre [M, K] x weight) and by the weight (dpre^T x x); the results that are
// null are left out
size_t product_grads_workspace_bytes(const ProductArgs &x, const ProductArgs &w);
hipError_t launch_product_grads(const ProductArgs &x, const ProductArgs &w, hipStream_t s);

// One file each: operands copied to LDS directly, or (_any) from any address
hipError_t launch_tiles_bf16(const ProductArgs &a, const ProductGrid &g, hipStream_t s);
hipError_t launch_tiles_bf16_any(const ProductArgs &a, const ProductGrid &g, hipStream_t s);
hipError_t launch_tiles_f32(const ProductArgs &a, const ProductGrid &g, hipStream_t s);
hipError_t launch_tiles_f32_any(const ProductArgs &a, const ProductGrid &g, hipStream_t s);
// Both products of a gradient in one launch (operands copied directly, tiles of 64)
hipError_t launch_pair_bf16(const ProductArgs &x, const ProductGrid &gx, const ProductArgs &w, const ProductGrid &gw,
                            bool x_first, hipStream_t s);
hipError_t launch_pair_f32(const ProductArgs &x, const ProductGrid &gx, const ProductArgs &w, const ProductGrid &gw,
                           bool x_first, hipStream_t s);

// Few rows: product_rows.hip, without a workspace
bool product_few_rows(const ProductArgs &a);
hipError_t launch_product_rows(const ProductArgs &a, hipStream_t s);

// The elementwise part of a backward and the sums over its rows
struct ProductActArgs {
    int64_t M, N;
    int dtype;
    bool gated;
    const void *dy;               // [M, N] at dy_ld
    int64_t dy_ld;
    const void *pre;              // linear [M, N] (null without an activation), gated [M, 2 N]
    bool pre_f32;
    int act;
    void *dpre;                   // like pre
    float *part;                  // workspace [product_act_rows, N or 2 N], null without dbias
    void *dbias;                  // [N or 2 N] (act dtype) or null
};
int64_t product_act_rows(int64_t M, int64_t N, int32_t dtype);
bool product_act_fits(const ProductActArgs &a);
hipError_t launch_product_act(const ProductActArgs &a, hipStream_t s);

// ---------------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------------
// The normal distribution's function Phi(v) = erfc(-v / sqrt 2) / 2.  erfc by the Chebyshev fit
// of Press, Teukolsky, Vetterling and Flannery (Numerical Recipes, 6.2), whose fractional error
// is below 1.2e-7 everywhere; its exponent is taken in two parts, so that the far tail keeps its
// relative accuracy too.
__device__ __forceinline__ float normal_cdf(float v) {
    const float z = fabsf(v) * 0.70710678118654752440f;
    const float t = rcp_fast(fmaf(0.5f, z, 1.f));
    float q = 0.17087277f;
    q = fmaf(q, t, -0.82215223f);
    q = fmaf(q, t, 1.48851587f);
    q = fmaf(q, t, -1.13520398f);
    q = fmaf(q, t, 0.27886807f);
    q = fmaf(q, t, -0.18628806f);
    q = fmaf(q, t, 0.09678418f);
    q = fmaf(q, t, 0.37409196f);
    q = fmaf(q, t, 1.00002368f);
    q = fmaf(q, t, -1.26551223f);
    // e^(-z^2 + q): the square and its product with log2(e) / 2 = kHalfLog2e + kHalfLog2eRest, each
    // with what its rounding left off
    constexpr float kHalfLog2e = 0.72134751f, kHalfLog2eRest = 9.62981495e-09f;
    const float v2 = v * v, x = kHalfLog2e * v2;
    const float rest = fmaf(kHalfLog2e, v2, -x) + fmaf(kHalfLog2eRest, v2, kHalfLog2e * fmaf(v, v, -v2));
    const float e = exp2_fast(-x) * exp2_fast(fmaf(kLog2eF, q, -rest));
    const float c = v2 < 3.0e4f ? 0.5f * t * e : 0.f;           // beyond, 0 x infinity; NaN takes the sum below
    return v != v ? v : (v < 0.f ? c : 1.f - c);
}

__device__ __forceinline__ float act_f32(float v, int act) {     // kActSilu or kActGelu
    const float c = act == kActSilu ? sigmoid_f32(v) : normal_cdf(v);
    return c == 0.f ? 0.f : v * c;                              // 0 at -infinity too
}
// The same for V values, with one branch for all of them: one for each, in the unrolled epilogue of
// a tile, took 24 us of a product's 185 (8192 x 2048 x 5632).
template <int V>
__device__ __forceinline__ void act_all(float (&v)[V], int act) {
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = act_f32(v[i], kActSilu);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = act_f32(v[i], kActGelu);
    }
}
// act(v) and, in *d, its derivative; kActSilu or kActGelu
__device__ __forceinline__ float act_d_f32(float v, int act, float *d) {
    const bool silu = act == kActSilu;
    const float c = silu ? sigmoid_f32(v) : normal_cdf(v);
    // c'(v): s (1 - s) or the normal density
    const float e = silu ? c * (1.f - c) : 0.39894228040143267794f * exp2_fast(-0.5f * kLog2eF * v * v);
    *d = e == 0.f ? c : fmaf(v, e, c);
    return c == 0.f ? 0.f : v * c;
}

// ---------------------------------------------------------------------------------
// Epilogues: V consecutive columns of one row
// ---------------------------------------------------------------------------------
template <typename T> constexpr int product_vec() { return 16 / (int)sizeof(T); }

// V values at p, or the first n of them (the rest 0), wherever p lies: global memory takes 16 bytes at
// any element's address
template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::type load_pack(const T *p, int n) {
    typename Pack<T, V>::type q;
    if (n >= V) {
        __builtin_memcpy(&q, p, sizeof(q));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = i < n ? p[i] : from_f32<T>(0.f);
    }
    return q;
}
template <typename T, int V>
__device__ __forceinline__ void load_some(const T *p, int n, float (&v)[V]) {
    unpack<T, V>(load_pack<T, V>(p, n), v);
}
template <typename T, int V>
__device__ __forceinline__ void store_some(T *p, int n, const float (&v)[V]) {
    if (n >= V) {
        typename Pack<T, V>::type q;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = from_f32<T>(v[i]);
        __builtin_memcpy(p, &q, sizeof(q));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

struct Epilogue {
    int64_t M, N;
    const void *bias, *residual;
    int64_t residual_ld;
    int act;
    void *y, *pre;
    bool pre_f32;
};

inline Epilogue epilogue_of(const ProductArgs &a) {
    return {a.M, a.N, a.bias, a.residual, a.residual_ld, a.act, a.y, a.pre, a.pre_f32};
}

// Columns n .. n + V - 1 of the bias, of its half `of_up` in a gated product, and of the residual's row
// m; zeros where there are none.  A tile reads those of all its rows before it stores any.
template <typename T, int V>
__device__ __forceinline__ void load_bias(const Epilogue &p, int64_t n, bool of_up, float (&b)[V]) {
    const int left = p.bias ? (int)min(p.N - n, (int64_t)V) : 0;
    load_some<T, V>(reinterpret_cast<const T *>(p.bias) + (of_up ? p.N : 0) + n, left, b);
}
template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::type load_residual(const Epilogue &p, int64_t m, int64_t n) {
    const int left = p.residual && m < p.M ? (int)min(p.N - n, (int64_t)V) : 0;
    return load_pack<T, V>(reinterpret_cast<const T *>(p.residual) + m * p.residual_ld + n, left);
}

template <typename T, int V>
__device__ __forceinline__ void store_pre(const Epilogue &p, int64_t at, int n, const float (&v)[V]) {
    if (sizeof(T) == 2 && p.pre_f32) store_some<float, V>(reinterpret_cast<float *>(p.pre) + at, n, v);
    else store_some<T, V>(reinterpret_cast<T *>(p.pre) + at, n, v);
}

// v: the product's values at row m, columns n .. n + V - 1; b and r: those of the bias and the residual
template <typename T, int V>
__device__ __forceinline__ void finish_linear(const Epilogue &p, int64_t m, int64_t n, const float (&b)[V],
                                              typename Pack<T, V>::type r, float (&v)[V]) {
    const int left = (int)min(p.N - n, (int64_t)V);
    if (left <= 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += b[i];
    if (p.pre) store_pre<T, V>(p, m * p.N + n, left, v);
    act_all<V>(v, p.act);
    if (p.residual) {
        float f[V];
        unpack<T, V>(r, f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += f[i];
    }
    store_some<T, V>(reinterpret_cast<T *>(p.y) + m * p.N + n, left, v);
}
template <typename T, int V>
__device__ __forceinline__ void finish_linear(const Epilogue &p, int64_t m, int64_t n, float (&v)[V]) {
    float b[V];
    load_bias<T, V>(p, n, false, b);
    finish_linear<T, V>(p, m, n, b, load_residual<T, V>(p, m, n), v);
}

// g and u: both products' values at row m, columns n .. n + V - 1 of each half; bg and bu: their biases
template <typename T, int V>
__device__ __forceinline__ void finish_gated(const Epilogue &p, int64_t m, int64_t n, const float (&bg)[V],
                                             const float (&bu)[V], float (&g)[V], float (&u)[V]) {
    const int left = (int)min(p.N - n, (int64_t)V);
    if (left <= 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        g[i] += bg[i];
        u[i] += bu[i];
    }
    if (p.pre) {
        store_pre<T, V>(p, 2 * m * p.N + n, left, g);
        store_pre<T, V>(p, (2 * m + 1) * p.N + n, left, u);
    }
    act_all<V>(g, p.act);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] *= u[i];
    store_some<T, V>(reinterpret_cast<T *>(p.y) + m * p.N + n, left, g);
}
template <typename T, int V>
__device__ __forceinline__ void finish_gated(const Epilogue &p, int64_t m, int64_t n, float (&g)[V], float (&u)[V]) {
    float bg[V], bu[V];
    load_bias<T, V>(p, n, false, bg);
    load_bias<T, V>(p, n, true, bu);
    finish_gated<T, V>(p, m, n, bg, bu, g, u);
}

}  // namespace ssd
