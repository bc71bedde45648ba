// The elementwise part of a product's backward, and the sums over rows that a bias' gradient
// is:
//
//     linear   dpre = dy act'(pre)
//     gated    d[g | u] = [dh u act'(g) | dh act(g)]
//     dbias    sum over rows of either (before it is rounded)
//
// dpre is rounded to the activations' type, in which the matrix units take it: one rounding of
// each term of dx and dweight, whose sums are float32.  A stream of 3 (linear) or 5 (gated)
// elements per result column; a wave takes 64 x 16 bytes of neighbouring columns and every 4th row of its
// workgroup's share, with one running sum a column, and a second kernel adds the workgroups'
// rows of sums in order, so results do not depend on scheduling.  Bound by memory: 8192 x (2 x 5632)
// in bfloat16 with pre in float32 146 us, 4.4 TB/s, and 5 for the sums (pre in bfloat16: 92, 5.0).
#include "product.h"

namespace ssd {

template <typename T, typename P, bool GATED>
__global__ __launch_bounds__(256) void product_act_kernel(ProductActArgs p, int64_t rows_each) {
    constexpr int V = product_vec<T>(), H = GATED ? 2 : 1;
    __shared__ float red[H][V][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t n = ((int64_t)blockIdx.x * 64 + lane) * V, cols = GATED ? 2 * p.N : p.N;
    const int left = (int)min(p.N - n, (int64_t)V);
    const int64_t first = (int64_t)blockIdx.y * rows_each, end = min(first + rows_each, p.M);
    float sum[H][V];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[h][i] = 0.f;
    const T *dy = reinterpret_cast<const T *>(p.dy) + n;
    const P *pre = reinterpret_cast<const P *>(p.pre) + n;
    T *dpre = reinterpret_cast<T *>(p.dpre) + n;
    if (left > 0)
#pragma unroll 2
        for (int64_t m = first + wave; m < end; m += 4) {
            float d[V];
            load_some<T, V>(dy + m * p.dy_ld, left, d);
            if constexpr (GATED) {
                float g[V], u[V];
                load_some<P, V>(pre + m * cols, left, g);
                load_some<P, V>(pre + m * cols + p.N, left, u);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float s;
                    const float h = act_d_f32(g[i], p.act, &s);
                    g[i] = d[i] * u[i] * s;
                    u[i] = d[i] * h;
                    sum[0][i] += g[i];
                    sum[1][i] += u[i];
                }
                store_some<T, V>(dpre + m * cols, left, g);
                store_some<T, V>(dpre + m * cols + p.N, left, u);
            } else {
                if (p.act != kActNone) {
                    float v[V];
                    load_some<P, V>(pre + m * cols, left, v);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float s;
                        act_d_f32(v[i], p.act, &s);
                        d[i] *= s;
                    }
                    store_some<T, V>(dpre + m * cols, left, d);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0][i] += d[i];
            }
        }
    if (!p.part) return;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        for (int w = 0; w < 4; ++w) {
            if (wave == w)
#pragma unroll
                for (int i = 0; i < V; ++i) red[h][i][lane] = (w ? red[h][i][lane] : 0.f) + sum[h][i];
            __syncthreads();
        }
        if (wave == 0)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < left) p.part[blockIdx.y * cols + h * p.N + n + i] = red[h][i][lane];
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void product_bias_kernel(const float *part, int rows, int64_t cols, T *out) {
    __shared__ float red[16][64];
    const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
    const float s = rows_sum<16>(part + min(col, cols - 1), rows, cols, red);
    if (threadIdx.x < 64 && col < cols) out[col] = from_f32<T>(s);
}

// Workgroups over the rows: about 2048 of 4 waves in all, 16 rows for each at least.
int64_t product_act_rows(int64_t M, int64_t N, int32_t dtype) {
    const int64_t w = dtype == 1 ? 512 : 256, across = (N + w - 1) / w;
    int64_t n = (2048 + across - 1) / across;
    if (n > (M + 15) / 16) n = (M + 15) / 16;
    return n;
}

static int64_t act_across(const ProductActArgs &a) {
    const int64_t w = a.dtype == 1 ? 512 : 256;
    return (a.N + w - 1) / w;
}

bool product_act_fits(const ProductActArgs &a) {
    return grid_fits(act_across(a), 256) && grid_fits((a.N * (a.gated ? 2 : 1) + 63) / 64, 1024);
}

// P: pre's type
template <typename T, typename P>
static void act_launch(const ProductActArgs &a, dim3 grid, int64_t rows_each, hipStream_t s) {
    if (a.gated) product_act_kernel<T, P, true><<<grid, 256, 0, s>>>(a, rows_each);
    else product_act_kernel<T, P, false><<<grid, 256, 0, s>>>(a, rows_each);
}

hipError_t launch_product_act(const ProductActArgs &a, hipStream_t s) {
    const int64_t blocks = product_act_rows(a.M, a.N, a.dtype), each = (a.M + blocks - 1) / blocks;
    const dim3 grid((uint32_t)act_across(a), (uint32_t)((a.M + each - 1) / each));
    if (a.dtype == 1 && !a.pre_f32) act_launch<bf16, bf16>(a, grid, each, s);
    else if (a.dtype == 1) act_launch<bf16, float>(a, grid, each, s);
    else act_launch<float, float>(a, grid, each, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dbias) return e;
    const int64_t cols = a.gated ? 2 * a.N : a.N;
    const uint32_t sums = (uint32_t)((cols + 63) / 64);
    if (a.dtype == 1) product_bias_kernel<bf16><<<sums, 1024, 0, s>>>(a.part, (int)grid.y, cols, (bf16 *)a.dbias);
    else product_bias_kernel<float><<<sums, 1024, 0, s>>>(a.part, (int)grid.y, cols, (float *)a.dbias);
    return hipGetLastError();
}

}  // namespace ssd
