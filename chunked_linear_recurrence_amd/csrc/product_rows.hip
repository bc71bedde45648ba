// The products of product.h for few rows (single tokens of a batch): a stream of the weight's rows,
// each read once, with nothing staged in LDS.
//
// A workgroup takes 16 rows of the weight (gated: 16 of g and the 16 of u beside them), or 32, and
// its waves a contiguous share of k each, so that even a weight of a few megabytes is on its way
// in a thousand waves at once.  A lane's 16 bytes are its fragment of the matrix units as they
// come from memory (row lane % 16, 8 or 4 values of k); x's fragments, 16 rows of x each, come
// from the caches the same way.  The waves' sums are added in wave order through LDS.
#include "product_tile.h"

namespace ssd {

template <typename T, ProductKind KIND, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void product_rows_kernel(ProductArgs p, Epilogue ep) {
    typedef typename Frag<T>::type F;
    constexpr int V = 16 / (int)sizeof(T), KS = kStepBytes / (int)sizeof(T), TILES = KIND == kGated ? 2 * NT : NT;
    constexpr int U = MT * TILES > 4 ? 1 : MT > 1 ? 2 : 4;       // steps whose loads are started together
    // Whether the next ones are on their way while these are multiplied, where few waves share a CU and
    // registers hold both: 48 rows of 6216 x (2 x 4200) 44.2 -> 38.1 us, 33 of 2048 x (2 x 5632) 17.4 ->
    // 14.9; one row of 4096 x (2 x 8192) 22.1 -> 24.1, so not for it.
    constexpr bool AHEAD = NT == 2 && (MT == 2 || MT == 3);
    __shared__ f32x4 sums[WAVES][MT][TILES][64];
    const int lane = threadIdx.x % 64, i16 = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t n0 = (int64_t)blockIdx.x * 16 * NT;
    const int64_t steps = (p.K + KS - 1) / KS, whole = p.K / KS;
    const int64_t first = steps * wave / WAVES, end = steps * (wave + 1) / WAVES;
    const T *x[MT], *b[TILES];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        x[i] = reinterpret_cast<const T *>(p.a.p) + min((int64_t)(16 * i + i16), p.M - 1) * p.a.ld + g * V;
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
        const int64_t row = min(n0 + 16 * (j % NT) + i16, p.N - 1) + (j / NT) * p.N;
        b[j] = reinterpret_cast<const T *>(p.b.p) + row * p.b.ld + g * V;
    }
    f32x4 acc[MT][TILES];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < TILES; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto load = [](const T *q) SSD_INLINE {
        F f;
        __builtin_memcpy(&f, q, 16);
        return f;
    };
    // the fragments of N steps
    auto fetch = [&](int64_t s, auto &fb, auto &fx) SSD_INLINE {
        constexpr int N = (int)(sizeof(fb) / sizeof(fb[0]));
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (s + q) * KS + h * (KS / 2);
#pragma unroll
                for (int j = 0; j < TILES; ++j) fb[q][h][j] = load(b[j] + k);
#pragma unroll
                for (int i = 0; i < MT; ++i) fx[q][h][i] = load(x[i] + k);
            }
    };
    auto products = [&](const auto &fb, const auto &fx) SSD_INLINE {
        constexpr int N = (int)(sizeof(fb) / sizeof(fb[0]));
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < TILES; ++j) acc[i][j] = multiply(fb[q][h][j], fx[q][h][i], acc[i][j]);
    };
    int64_t s = first;
    const int64_t full = min(end, whole);
    if constexpr (AHEAD) {
        F fb[2][U][2][TILES], fx[2][U][2][MT];
        if (s + U <= full) {
            fetch(s, fb[0], fx[0]);
            s += U;
            while (s + 2 * U <= full) {
                fetch(s, fb[1], fx[1]);
                __builtin_amdgcn_sched_barrier(0);
                products(fb[0], fx[0]);
                fetch(s + U, fb[0], fx[0]);
                __builtin_amdgcn_sched_barrier(0);
                products(fb[1], fx[1]);
                s += 2 * U;
            }
            products(fb[0], fx[0]);
        }
    }
    for (; s + U <= full; s += U) {
        F fb[U][2][TILES], fx[U][2][MT];
        fetch(s, fb, fx);
        products(fb, fx);
    }
    for (; U > 1 && s < full; ++s) {
        F fb[1][2][TILES], fx[1][2][MT];
        fetch(s, fb, fx);
        products(fb, fx);
    }
    if (s < end) {                                               // the step that K ends in
        auto some = [&](const T *q, int64_t k) SSD_INLINE {
            const int64_t have = p.K - k - g * V;
            T v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = e < have ? q[k + e] : from_f32<T>(0.f);
            F f;
            __builtin_memcpy(&f, v, 16);
            return f;
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = s * KS + h * (KS / 2);
            F fb[TILES];
#pragma unroll
            for (int j = 0; j < TILES; ++j) fb[j] = some(b[j], k);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const F fx = some(x[i], k);
#pragma unroll
                for (int j = 0; j < TILES; ++j) acc[i][j] = multiply(fb[j], fx, acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < TILES; ++j) sums[wave][i][j][lane] = acc[i][j];
    __syncthreads();
    // results of (16 rows of x, 16 columns) by one wave each: lane (i16, g) has row i16, columns 4 g ..
    for (int t = wave; t < MT * NT; t += WAVES) {
        const int i = t / NT, j = t % NT;
        auto total = [&](int tile, float (&v)[4]) SSD_INLINE {
            f32x4 r = sums[0][i][tile][lane];
            for (int w = 1; w < WAVES; ++w) r += sums[w][i][tile][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = r[e];
        };
        const int64_t m = 16 * i + i16, n = n0 + 16 * j + 4 * g;
        if (m >= p.M) continue;
        float v[4];
        total(j, v);
        if constexpr (KIND == kGated) {
            float u[4];
            total(NT + j, u);
            finish_gated<T, 4>(ep, m, n, v, u);
        } else {
            finish_linear<T, 4>(ep, m, n, v);
        }
    }
}

// Up to 32 rows; up to 48 of a weight of many rows, which workgroups take 32 at a time; up to 64 of a
// small weight: beyond, tiles share x's reads, which here every workgroup makes for itself.  Kernels
// among others, weights from memory, us here and in tiles, bfloat16: 2048 x 4096 32 rows 9.1 and 13.8, 33
// 10.4 and 13.7; 4096 x 4096 32 rows 14.6 and 19.4, 33 16.9 and 19.3, 49 22.4 and 19.6; 2048 x (2 x 5632)
// 48 rows 16.8 and 25.4, 49 20.6 and 25.3; 4096 x 4160 48 rows 22.5 and 23.4, 64 25.8 and 23.4; 1536 x 768
// 64 rows 10.2 and 10.0, 1024 x 1024 7.9 and 11.5.  Float32: 2048 x 4096 32 rows 15.3 and 21.5, 1024 x
// 1024 64 rows 12.5 and 11.4.  The edges are those of bfloat16 and do not look at k: to either side of
// them the other way is quicker at 33 to 48 rows of up to 4096 (2048 x (2 x 4096) 12.1 and 25.7), at 49
// to 64 of a short k, and in tiles at 4096 x (2 x 4160) from 32 rows on (25.9 and 23.9) and for
// 33 rows of a small float32 weight (2048 x (2 x 1024) 28.4 and 18.2).
bool product_few_rows(const ProductArgs &a) {
    if (a.a_rows || a.b_rows) return false;
    return a.M <= SSD_PRODUCT_FEW_ROWS || (a.M <= 48 && a.N > 4096) ||
           (a.M <= 64 && a.N * a.K <= (INT64_C(1) << 22));
}

// 16 rows of the weight a workgroup and up to 16 waves for them up to 4096 rows, a workgroup for each
// CU, else 32 rows, which halves the reads of x, and 4 waves, 8 for 33 to 48 rows.  16 and 32 rows a
// workgroup, bfloat16: 32 rows of 2048 x 4096 9.1 us and 11.1, of 2048 x 4160 14.1 and 11.0, of 2048 x (2 x
// 4096) 11.8 and 15.1, of 2048 x (2 x 4160) 18.9 and 15.5; one row of 2048 x 4096 6.0 and 8.4, of 4160
// 8.7 and 8.4; float32, one row of 2048 x 4096 8.8 and 14.3, of 5632 13.4 and 14.2.  4 and 8 waves by 32:
// 48 rows of 2048 x (2 x 5632) 17.6 and 16.8 (float32 31.9 and 36.0), 32 rows 15.2 and 15.7.
template <typename T, ProductKind KIND, int MT>
static hipError_t rows_launch(const ProductArgs &a, hipStream_t s) {
    const Epilogue ep = epilogue_of(a);
    constexpr int WAVES = MT == 1 ? 16 : MT == 2 ? 8 : 4, WIDE = MT == 3 ? 8 : 4;
    if (a.N <= 4096) product_rows_kernel<T, KIND, MT, 1, WAVES><<<(uint32_t)((a.N + 15) / 16), 64 * WAVES, 0, s>>>(a, ep);
    else product_rows_kernel<T, KIND, MT, 2, WIDE><<<(uint32_t)((a.N + 31) / 32), 64 * WIDE, 0, s>>>(a, ep);
    return hipGetLastError();
}

template <typename T>
static hipError_t rows_by_m(const ProductArgs &a, hipStream_t s) {
    const bool gated = a.kind == kGated;
    if (a.M <= 16) return gated ? rows_launch<T, kGated, 1>(a, s) : rows_launch<T, kLinear, 1>(a, s);
    if (a.M <= 32) return gated ? rows_launch<T, kGated, 2>(a, s) : rows_launch<T, kLinear, 2>(a, s);
    if (a.M <= 48) return gated ? rows_launch<T, kGated, 3>(a, s) : rows_launch<T, kLinear, 3>(a, s);
    return gated ? rows_launch<T, kGated, 4>(a, s) : rows_launch<T, kLinear, 4>(a, s);
}

hipError_t launch_product_rows(const ProductArgs &a, hipStream_t s) {
    return a.dtype == 1 ? rows_by_m<bf16>(a, s) : rows_by_m<float>(a, s);
}

}  // namespace ssd
