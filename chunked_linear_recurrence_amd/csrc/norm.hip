// Layer norm of rows of D channels, and its backward:
//
//     mean = sum x / D;  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps);  xhat = (x - mean) rstd
//     y  = xhat w + b
//     dx = rstd (g - sum(g) / D - xhat sum(g xhat) / D),  g = dy w
//     dw = sum over rows of dy xhat;  db = sum over rows of dy
//
// A stream of 2 elements in the forward and 3 in the backward per element; nothing else can
// bound it, so a row is read once and held in registers: the variance is summed about the
// finished mean (no difference of large sums), and the backward forms both row sums, dx and
// its share of dw and db from the same copy.  A row belongs to 1, 4 or 16 waves, the fewest
// whose registers hold it; rows that 16 waves cannot hold are read again for each pass.
// dw and db: each workgroup walks many rows with one running sum per column in float32,
// leaves one row of partial sums, and a second kernel adds those rows in order, so results
// do not depend on scheduling.  32768 rows of 2048 channels in bfloat16: 50 us forward
// (5.4 TB/s), 84 + 5 us backward (4.8).  2048 rows of 32768, which no registers hold: 165 us
// forward, 156 + 105 + 22 backward, where the copy rate gives 56 and 84.
#include "ssd_block.h"

namespace ssd {

constexpr int kNormBwdBlocks = 512;    // workgroups (rows of partial sums) of the backward at most
constexpr int kNormFwdBlocks = 1024;   // workgroups of 4 waves of the forward at most

// Sum over the 64 lanes, the same in every lane: 4 steps within rows of 16 lanes on the vector
// units' own lane permutations, then the 4 rows' sums by way of scalar registers.  (Shuffles
// through LDS wait for it at each of 6 steps.)
template <int CTRL>
__device__ __forceinline__ float permuted(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += permuted<0xb1>(v);       // lanes 1 apart
    v += permuted<0x4e>(v);       // 2 apart
    v += permuted<0x141>(v);      // the other 4 of 8, mirrored
    v += permuted<0x140>(v);      // the other 8 of 16, mirrored
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Sums over the WPR waves that share a row (WPR > 1: every wave of the workgroup).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x / 64;
        __syncthreads();                       // the previous sum has been read
        if (threadIdx.x % 64 == 0) red[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) v += red[k];
    }
    return v;
}

template <int WPR> constexpr int norm_threads() { return WPR == 16 ? 1024 : 256; }
template <int WPR> constexpr bool norm_ahead() { return WPR < 16; }           // 1024 threads leave 128 registers each
template <int WPR> constexpr int norm_rows() { return WPR == 1 ? 4 : 1; }     // rows a workgroup holds at a time

template <typename T, int V>
__device__ __forceinline__ float pick(const typename Pack<T, V>::type &p, int i) {
    if constexpr (V == 1) return to_f32(p);
    else return (float)p[i];
}

template <int V>
__device__ __forceinline__ void load_param(const float *p, int c, float none, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p ? p[c + i] : none;
}

// A row's K accesses of this thread; those past the row are left alone.
template <typename T, int V, int K, int WPR>
__device__ __forceinline__ void load_row(const T *x, int D, int tid, typename Pack<T, V>::type (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * 64 * WPR + tid) * V;
        if (c < D) v[k] = *reinterpret_cast<const typename Pack<T, V>::type *>(x + c);
    }
}

// A workgroup walks many rows with weight and bias in registers (read per row they are four
// times a bfloat16 row's own traffic) and, where registers allow, the next row on its way while
// one is reduced: 32768 rows of 2048 channels take 50 us, against 71 with a row a wave.
template <typename T, int V, int K, int WPR>
__global__ __launch_bounds__(norm_threads<WPR>()) void norm_fwd_kernel(NormArgs a) {
    __shared__ float red[16];
    typedef typename Pack<T, V>::type P;
    constexpr int R = norm_rows<WPR>();
    const int tid = WPR == 1 ? threadIdx.x % 64 : threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * R + (WPR == 1 ? threadIdx.x / 64 : 0), by = (int64_t)gridDim.x * R;
    const T *x = reinterpret_cast<const T *>(a.x);
    P v[K] = {}, next[K] = {};
    if (first < a.rows) load_row<T, V, K, WPR>(x + first * a.x_stride, a.D, tid, next);
    float w[K][V], b[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * 64 * WPR + tid) * V;
        load_param<V>(c < a.D ? a.w : nullptr, c, 1.f, w[k]);
        load_param<V>(c < a.D ? a.bias : nullptr, c, 0.f, b[k]);
    }
    for (int64_t row = first; row < a.rows; row += by) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = next[k];
        if (norm_ahead<WPR>() && row + by < a.rows) load_row<T, V, K, WPR>(x + (row + by) * a.x_stride, a.D, tid, next);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * 64 * WPR + tid) * V < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) s += pick<T, V>(v[k], i);
        const float mean = row_sum<WPR>(s, red) / a.D;
        s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * 64 * WPR + tid) * V < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = pick<T, V>(v[k], i) - mean;
                    s = fmaf(d, d, s);
                }
        const float rstd = 1.f / sqrtf(row_sum<WPR>(s, red) / a.D + a.eps);
        T *y = reinterpret_cast<T *>(a.y) + row * a.D;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * 64 * WPR + tid) * V;
            if (c < a.D) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf((pick<T, V>(v[k], i) - mean) * rstd, w[k][i], b[k][i]);
                store_f32<T, V>(y + c, o);
            }
        }
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (!norm_ahead<WPR>() && row + by < a.rows) load_row<T, V, K, WPR>(x + (row + by) * a.x_stride, a.D, tid, next);
    }
}

// Rows wider than registers: one workgroup a row, three passes over it.
template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(NormArgs a) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride;
    T *y = reinterpret_cast<T *>(a.y) + row * a.D;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) s += to_f32(x[c]);
    const float mean = row_sum<16>(s, red) / a.D;
    s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(row_sum<16>(s, red) / a.D + a.eps);
    for (int c = threadIdx.x; c < a.D; c += 1024)
        y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w ? a.w[c] : 1.f, a.bias ? a.bias[c] : 0.f));
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename T, int V, int K, int WPR>
__global__ __launch_bounds__(norm_threads<WPR>()) void norm_bwd_kernel(NormArgs a) {
    __shared__ float red[16];
    __shared__ float cols[WPR == 1 ? 2 * 64 * V * K : 1];
    typedef typename Pack<T, V>::type P;
    constexpr int R = norm_rows<WPR>();
    const int wave = threadIdx.x / 64;
    const int tid = WPR == 1 ? threadIdx.x % 64 : threadIdx.x;
    float dw[K][V], db[K][V], w[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * 64 * WPR + tid) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dw[k][i] = db[k][i] = 0.f;
            w[k][i] = (a.w && c < a.D) ? a.w[c + i] : 1.f;
        }
    }
    const T *x = reinterpret_cast<const T *>(a.x), *dy = reinterpret_cast<const T *>(a.dy);
    const int64_t first = (int64_t)blockIdx.x * R + (WPR == 1 ? wave : 0), by = (int64_t)gridDim.x * R;
    P xv[K] = {}, gv[K] = {}, xn[K] = {}, gn[K] = {};
    float mean_n = 0.f, rstd_n = 0.f;
    auto fetch = [&](int64_t row) {
        load_row<T, V, K, WPR>(x + row * a.x_stride, a.D, tid, xn);
        load_row<T, V, K, WPR>(dy + row * a.dy_stride, a.D, tid, gn);
        mean_n = a.mean[row];
        rstd_n = a.rstd[row];
    };
    if (first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += by) {
        const float mean = mean_n, rstd = rstd_n;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xv[k] = xn[k];
            gv[k] = gn[k];
        }
        if (norm_ahead<WPR>() && row + by < a.rows) fetch(row + by);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if ((k * 64 * WPR + tid) * V < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float h = (pick<T, V>(xv[k], i) - mean) * rstd, d = pick<T, V>(gv[k], i), g = d * w[k][i];
                    s1 += g;
                    s2 = fmaf(g, h, s2);
                    dw[k][i] = fmaf(d, h, dw[k][i]);
                    db[k][i] += d;
                }
        }
        s1 = row_sum<WPR>(s1, red) / a.D;
        s2 = row_sum<WPR>(s2, red) / a.D;
        T *dx = reinterpret_cast<T *>(a.dx) + row * a.D;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * 64 * WPR + tid) * V;
            if (c < a.D) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float h = (pick<T, V>(xv[k], i) - mean) * rstd, g = pick<T, V>(gv[k], i) * w[k][i];
                    o[i] = rstd * (g - s1 - h * s2);
                }
                store_f32<T, V>(dx + c, o);
            }
        }
        if (!norm_ahead<WPR>() && row + by < a.rows) fetch(row + by);
    }
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.D;
    if constexpr (WPR == 1) {
        // the 4 waves add their sums in wave order
        constexpr int M = 64 * V * K;
        for (int q = 0; q < 4; ++q) {
            if (wave == q) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int at = (k * V + i) * 64 + tid;          // lanes side by side
                        cols[at] = (q ? cols[at] : 0.f) + dw[k][i];
                        cols[M + at] = (q ? cols[M + at] : 0.f) + db[k][i];
                    }
            }
            __syncthreads();
        }
        for (int m = threadIdx.x; m < M; m += 256) {
            const int l = m % 64, ki = m / 64;
            const int c = ((ki / V) * 64 + l) * V + ki % V;
            if (c < a.D) {
                part[c] = cols[m];
                part[a.D + c] = cols[M + m];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * 64 * WPR + tid) * V;
            if (c < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    part[c + i] = dw[k][i];
                    part[a.D + c + i] = db[k][i];
                }
        }
    }
}

// Rows wider than registers: row sums in one pass and dx in a second ...
template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormArgs a) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride;
    const T *dy = reinterpret_cast<const T *>(a.dy) + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float g = to_f32(dy[c]) * (a.w ? a.w[c] : 1.f);
        s1 += g;
        s2 = fmaf(g, (to_f32(x[c]) - mean) * rstd, s2);
    }
    s1 = row_sum<16>(s1, red) / a.D;
    s2 = row_sum<16>(s2, red) / a.D;
    T *dx = reinterpret_cast<T *>(a.dx) + row * a.D;
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float g = to_f32(dy[c]) * (a.w ? a.w[c] : 1.f);
        dx[c] = from_f32<T>(rstd * (g - s1 - (to_f32(x[c]) - mean) * rstd * s2));
    }
}

// ... and the columns' sums over blockIdx.y's share of the rows in a kernel of its own.
template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_cols_kernel(NormArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D) return;
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = to_f32(reinterpret_cast<const T *>(a.dy)[row * a.dy_stride + c]);
        dw = fmaf(d, (to_f32(reinterpret_cast<const T *>(a.x)[row * a.x_stride + c]) - a.mean[row]) * a.rstd[row], dw);
        db += d;
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.D;
    part[c] = dw;
    part[a.D + c] = db;
}

__global__ __launch_bounds__(1024) void norm_bwd_sum_kernel(const float *part, int rows, int D, float *dw, float *db) {
    __shared__ float red[16][64];
    const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x % 64, cols = 2 * (int64_t)D;
    const float s = rows_sum<16>(part + min(col, cols - 1), rows, cols, red);
    if (threadIdx.x >= 64 || col >= cols) return;
    if (col < D) {
        if (dw) dw[col] = s;
    } else if (db) db[col - D] = s;
}

int64_t norm_bwd_blocks(int64_t rows) { return rows < kNormBwdBlocks ? rows : kNormBwdBlocks; }

template <typename T, int V, int K, int WPR>
static hipError_t norm_fwd_t(const NormArgs &a, hipStream_t s) {
    constexpr int R = norm_rows<WPR>(), cap = kNormFwdBlocks / (WPR == 16 ? 4 : 1);
    int64_t n = (a.rows + R - 1) / R;
    if (n > cap) n = cap;
    norm_fwd_kernel<T, V, K, WPR><<<(uint32_t)n, norm_threads<WPR>(), 0, s>>>(a);
    return hipGetLastError();
}

// Workgroups of the sums over rows; rows that registers hold have far fewer columns than a launch.
static int64_t norm_sum_blocks(const NormArgs &a) { return (2 * (int64_t)a.D + 63) / 64; }
static bool norm_sum_fits(const NormArgs &a) { return (!a.dw && !a.db) || grid_fits(norm_sum_blocks(a), 1024); }

static hipError_t norm_bwd_sum(const NormArgs &a, int64_t blocks, hipStream_t s) {
    if (!a.dw && !a.db) return hipSuccess;
    norm_bwd_sum_kernel<<<(uint32_t)norm_sum_blocks(a), 1024, 0, s>>>(a.part, (int)blocks, a.D, a.dw, a.db);
    return hipGetLastError();
}

template <typename T, int V, int K, int WPR>
static hipError_t norm_bwd_t(const NormArgs &a, hipStream_t s) {
    constexpr int R = norm_rows<WPR>();
    int64_t n = (a.rows + R - 1) / R;
    const int64_t cap = norm_bwd_blocks(a.rows);
    if (n > cap) n = cap;
    norm_bwd_kernel<T, V, K, WPR><<<(uint32_t)n, norm_threads<WPR>(), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : norm_bwd_sum(a, n, s);
}

template <typename T>
static hipError_t norm_fwd_wide_t(const NormArgs &a, hipStream_t s) {
    if (!grid_fits(a.rows, 1024)) return hipErrorInvalidValue;
    norm_fwd_wide_kernel<T><<<(uint32_t)a.rows, 1024, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
static hipError_t norm_bwd_wide_t(const NormArgs &a, hipStream_t s) {
    if (!grid_fits(a.rows, 1024) || !norm_sum_fits(a)) return hipErrorInvalidValue;
    norm_bwd_wide_kernel<T><<<(uint32_t)a.rows, 1024, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!a.dw && !a.db)) return e;
    const int64_t n = norm_bwd_blocks(a.rows);
    norm_bwd_cols_kernel<T><<<dim3((a.D + 255) / 256, (uint32_t)n), 256, 0, s>>>(a);
    e = hipGetLastError();
    return e != hipSuccess ? e : norm_bwd_sum(a, n, s);
}

static bool at16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// The fewest waves whose registers hold a row of D channels, V at a time.
#define NORM_VEC(DIR, T, V)                                                        \
    do {                                                                           \
        if (a.D <= 64 * V) return norm_##DIR##_t<T, V, 1, 1>(a, s);                \
        if (a.D <= 64 * V * 2) return norm_##DIR##_t<T, V, 2, 1>(a, s);            \
        if (a.D <= 64 * V * 4) return norm_##DIR##_t<T, V, 4, 1>(a, s);            \
        if (a.D <= 256 * V * 2) return norm_##DIR##_t<T, V, 2, 4>(a, s);           \
        if (a.D <= 256 * V * 4) return norm_##DIR##_t<T, V, 4, 4>(a, s);           \
        if (a.D <= 1024 * V * 2) return norm_##DIR##_t<T, V, 2, 16>(a, s);         \
    } while (0)
#define NORM_ONE(DIR, T)                                                           \
    do {                                                                           \
        if (a.D <= 256) return norm_##DIR##_t<T, 1, 4, 1>(a, s);                   \
        if (a.D <= 1024) return norm_##DIR##_t<T, 1, 4, 4>(a, s);                  \
        if (a.D <= 2048) return norm_##DIR##_t<T, 1, 8, 4>(a, s);                  \
        if (a.D <= 8192) return norm_##DIR##_t<T, 1, 8, 16>(a, s);                 \
    } while (0)

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s) {
    const int V = a.dtype == 1 ? 8 : 4;
    const bool vec = a.D % V == 0 && a.x_stride % V == 0 && at16(a.x) && at16(a.y);
    if (a.dtype == 1) {
        if (vec) NORM_VEC(fwd, bf16, 8);
        NORM_ONE(fwd, bf16);
        return norm_fwd_wide_t<bf16>(a, s);
    }
    if (vec) NORM_VEC(fwd, float, 4);
    NORM_ONE(fwd, float);
    return norm_fwd_wide_t<float>(a, s);
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t s) {
    const int V = a.dtype == 1 ? 8 : 4;
    const bool vec = a.D % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 && at16(a.x) && at16(a.dy) && at16(a.dx);
    if (a.dtype == 1) {
        if (vec) NORM_VEC(bwd, bf16, 8);
        NORM_ONE(bwd, bf16);
        return norm_bwd_wide_t<bf16>(a, s);
    }
    if (vec) NORM_VEC(bwd, float, 4);
    NORM_ONE(bwd, float);
    return norm_bwd_wide_t<float>(a, s);
}

}  // namespace ssd
