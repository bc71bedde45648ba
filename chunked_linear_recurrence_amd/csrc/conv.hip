// Short causal convolution over the tokens of each channel, with an optional SiLU:
//
//     pre_t = bias + sum_j w[j] x_{t - (W-1) + j},  j = 0..W-1;   y_t = pre_t or pre_t * sigmoid(pre_t)
//
// Tokens before the first come from the carried state (the last W-1 inputs, oldest first)
// or are zero.  Its backward, with dpre_t = dy_t d(pre_t):
//
//     dx_t = sum_j w[j] dpre_{t + (W-1) - j};  dw[j] = sum_{b,t} dpre_t x_{t - (W-1) + j};  dbias = sum dpre_t
//
// Both are streams: 2 W + 6 operations per element against 2 elements moved (3 in the
// backward), far below what the vector units do, so the layout serves the loads: a thread
// owns V consecutive channels (16 bytes where addresses allow it) and walks TS tokens with
// the last W-1 inputs in registers, so that an input is read from memory once, plus W-1
// tokens per TS that the caches hold.
#include "ssd_block.h"

namespace ssd {

constexpr int kConvWaves = 4;       // token segments per workgroup, one wave each
constexpr int kConvBwdTokens = 32;  // tokens per wave in the backward

struct ConvUnit {
    int64_t b;
    int t0, c;
};

// Workgroup -> (batch row, first token of this wave, first channel of this thread).
template <int V>
__device__ __forceinline__ ConvUnit conv_unit(int L, int C, int TS) {
    const int nct = (C + 64 * V - 1) / (64 * V);
    const int ntb = (L + kConvWaves * TS - 1) / (kConvWaves * TS);
    const int ct = blockIdx.x % nct;
    const int64_t r = blockIdx.x / nct;
    ConvUnit q;
    q.b = r / ntb;
    q.t0 = ((int)(r % ntb) * kConvWaves + threadIdx.x / 64) * TS;
    q.c = (ct * 64 + threadIdx.x % 64) * V;
    return q;
}

// Input t of a row of `len` tokens as float32; t < 0 reaches into the carried state.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_input(const ConvArgs &a, int64_t b, int t, int len, int c, float (&v)[V]) {
    if (t >= 0 && t < len) {
        load_f32<T, V>(row_of<T>(a.x, b, t) + c, v);
    } else if (t < 0 && a.init) {
        load_f32<T, V>(reinterpret_cast<const T *>(a.init) + (b * (W - 1) + (t + W - 1)) * a.C + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <int W, int V>
__device__ __forceinline__ void conv_weights(const ConvArgs &a, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.w[(int64_t)(c + i) * W + j];
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
    }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int TS) {
    const ConvUnit q = conv_unit<V>(a.L, a.C, TS);
    if (q.c >= a.C || q.t0 >= a.L) return;
    const int len = row_length(a.lengths, q.b, a.L);
    const bool silu = (a.flags & SSD_FLAG_SILU) != 0;
    float w[W][V], bias[V], win[W][V];
    conv_weights<W, V>(a, q.c, w, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q.b, q.t0 - (W - 1) + k, len, q.c, win[k]);
    // The state of the row's last token: the thread that holds the row's start writes it, as
    // it alone reads the incoming state, which may be the same memory.
    if (q.t0 == 0 && a.final_state) {
        float f[W - 1][V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q.b, len - (W - 1) + k, len, q.c, f[k]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_f32<T, V>(reinterpret_cast<T *>(a.final_state) + (q.b * (W - 1) + k) * a.C + q.c, f[k]);
    }
    const int t1 = min(q.t0 + TS, a.L);
    T *y = reinterpret_cast<T *>(a.y) + (q.b * a.L + q.t0) * (int64_t)a.C + q.c;
#pragma unroll 4
    for (int t = q.t0; t < t1; ++t, y += a.C) {
        float o[V];
        if (t < len) {
            load_f32<T, V>(row_of<T>(a.x, q.b, t) + q.c, win[W - 1]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) s = fmaf(w[j][i], win[j][i], s);
                o[i] = silu ? silu_f32(s) : s;
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = 0.f;
        }
        store_f32<T, V>(y, o);
    }
}

// One token: y from the state and x, and the state moved on by one (in place or not).
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a) {
    const int nt = (a.C + V - 1) / V;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.batch * nt) return;
    const int64_t b = k / nt;
    const int c = (int)(k % nt) * V;
    float w[W][V], bias[V], win[W][V], o[V];
    conv_weights<W, V>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        load_f32<T, V>(reinterpret_cast<const T *>(a.init) + (b * (W - 1) + j) * a.C + c, win[j]);
    load_f32<T, V>(reinterpret_cast<const T *>(a.x.p) + b * a.x.bs + c, win[W - 1]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float s = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[j][i], win[j][i], s);
        o[i] = (a.flags & SSD_FLAG_SILU) ? silu_f32(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        store_f32<T, V>(reinterpret_cast<T *>(a.final_state) + (b * (W - 1) + j) * a.C + c, win[j + 1]);
    store_f32<T, V>(reinterpret_cast<T *>(a.y) + b * a.C + c, o);
}

// Backward.  A wave of tokens [t0, t1) recomputes pre and dpre for [t0, t1 + W-1) and writes
// dx for its own tokens (the wave at the row's start also the W-1 positions of the carried
// state); dw and dbias are summed over its own tokens only.  The sums of the workgroup's
// waves meet in LDS and leave as one row of partial sums.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int TS) {
    __shared__ float red[kConvWaves - 1][(W + 1) * V][64];
    const ConvUnit q = conv_unit<V>(a.L, a.C, TS);
    const bool live = q.c < a.C && q.t0 < a.L;
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (live) {
        const int len = row_length(a.lengths, q.b, a.L);
        const bool silu = (a.flags & SSD_FLAG_SILU) != 0;
        float w[W][V], bias[V], win[W][V], dp[W][V];       // dp[j] = dpre of token s - j
        conv_weights<W, V>(a, q.c, w, bias);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q.b, q.t0 - (W - 1) + k, len, q.c, win[k]);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) dp[j][i] = 0.f;
        const int t1 = min(q.t0 + TS, a.L);
        const int first = q.t0 == 0 ? -(W - 1) : q.t0;
#pragma unroll 2
        for (int s = q.t0; s < t1 + W - 1; ++s) {
#pragma unroll
            for (int j = W - 1; j > 0; --j)
#pragma unroll
                for (int i = 0; i < V; ++i) dp[j][i] = dp[j - 1][i];
            if (s < len) {
                float g[V];
                load_f32<T, V>(row_of<T>(a.x, q.b, s) + q.c, win[W - 1]);
                load_f32<T, V>(row_of<T>(a.dy, q.b, s) + q.c, g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][i], win[j][i], p);
                    dp[0][i] = silu ? g[i] * dsilu_f32(p) : g[i];
                }
                if (s < t1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        db[i] += dp[0][i];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fmaf(dp[0][i], win[j][i], dw[j][i]);
                    }
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) dp[0][i] = 0.f;
            }
            const int t = s - (W - 1);
            if (t < first) continue;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) o[i] = fmaf(w[j][i], dp[j][i], o[i]);
            }
            const int f = t - (len - (W - 1));             // this input's place in the final state
            if (a.dfinal && f >= 0 && f < W - 1) {
                float g[V];
                load_f32<T, V>(reinterpret_cast<const T *>(a.dfinal) + (q.b * (W - 1) + f) * a.C + q.c, g);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] += g[i];
            }
            if (t >= 0)
                store_f32<T, V>(reinterpret_cast<T *>(a.dx) + (q.b * a.L + t) * (int64_t)a.C + q.c, o);
            else if (a.dinit)
                store_f32<T, V>(reinterpret_cast<T *>(a.dinit) + (q.b * (W - 1) + (t + W - 1)) * a.C + q.c, o);
        }
    }
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) red[wave - 1][j * V + i][lane] = dw[j][i];
            red[wave - 1][W * V + i][lane] = db[i];
        }
    }
    __syncthreads();
    if (wave == 0 && q.c < a.C) {
#pragma unroll
        for (int k = 0; k < kConvWaves - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][i] += red[k][j * V + i][lane];
                db[i] += red[k][W * V + i][lane];
            }
        const int nct = (a.C + 64 * V - 1) / (64 * V);
        float *o = a.part + (int64_t)(blockIdx.x / nct) * (W + 1) * a.C + q.c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) o[(int64_t)j * a.C + i] = dw[j][i];
            o[(int64_t)W * a.C + i] = db[i];
        }
    }
}

// dw[c][j] and dbias[c] from the rows of partial sums [rows, W+1, C].
__global__ __launch_bounds__(1024) void conv_bwd_sum_kernel(const float *part, int64_t rows, int C, int W, float *dw,
                                                            float *dbias) {
    __shared__ float red[16][64];
    const int64_t cols = (int64_t)(W + 1) * C, col = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
    const float s = rows_sum<16>(part + min(col, cols - 1), rows, cols, red);
    if (threadIdx.x >= 64 || col >= cols) return;
    const int j = (int)(col / C), c = (int)(col % C);
    if (j < W) dw[(int64_t)c * W + j] = s;
    else if (dbias) dbias[c] = s;
}

bool conv_supported(int W) { return W >= 2 && W <= 4; }

int64_t conv_bwd_rows(int64_t batch, int64_t L) {
    const int64_t per = kConvWaves * kConvBwdTokens;
    return batch * ((L + per - 1) / per);
}

// 16-byte accesses need every tensor's start, and every row's, on a 16-byte boundary.
static bool vector_rows(const View &v, int V, int64_t e) {
    return ((uintptr_t)v.p & 15u) == 0 && v.bs % V == 0 && v.ts % V == 0 && V * e == 16;
}
static bool at16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <typename T, int W, int V>
static hipError_t conv_fwd_t(const ConvArgs &a, hipStream_t s) {
    const int TS = 16;
    const int64_t nct = (a.C + 64 * V - 1) / (64 * V), ntb = (a.L + kConvWaves * TS - 1) / (kConvWaves * TS);
    const int64_t n = a.batch * ntb * nct;
    if (n > INT32_MAX) return hipErrorInvalidValue;
    conv_fwd_kernel<T, W, V><<<(uint32_t)n, 256, 0, s>>>(a, TS);
    return hipGetLastError();
}

template <typename T, int W, int V>
static hipError_t conv_step_t(const ConvArgs &a, hipStream_t s) {
    const int64_t n = (a.batch * ((a.C + V - 1) / V) + 255) / 256;
    if (n > INT32_MAX) return hipErrorInvalidValue;
    conv_step_kernel<T, W, V><<<(uint32_t)n, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int W, int V>
static hipError_t conv_bwd_t(const ConvArgs &a, hipStream_t s) {
    const int64_t nct = (a.C + 64 * V - 1) / (64 * V), rows = conv_bwd_rows(a.batch, a.L);
    if (rows * nct > INT32_MAX) return hipErrorInvalidValue;
    conv_bwd_kernel<T, W, V><<<(uint32_t)(rows * nct), 256, 0, s>>>(a, kConvBwdTokens);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)(W + 1) * a.C;
    conv_bwd_sum_kernel<<<(uint32_t)((cols + 63) / 64), 1024, 0, s>>>(a.part, rows, a.C, W, a.dw, a.dbias);
    return hipGetLastError();
}

#define CONV_PICK(FN, T, V)                          \
    switch (a.W) {                                   \
        case 2: return FN<T, 2, V>(a, s);            \
        case 3: return FN<T, 3, V>(a, s);            \
        case 4: return FN<T, 4, V>(a, s);            \
        default: return hipErrorInvalidValue;        \
    }
#define CONV_DISPATCH(FN, VEC)                       \
    if (a.dtype == 1) {                              \
        if (VEC(8, 2)) { CONV_PICK(FN, bf16, 8) }    \
        CONV_PICK(FN, bf16, 1)                       \
    }                                                \
    if (VEC(4, 4)) { CONV_PICK(FN, float, 4) }       \
    CONV_PICK(FN, float, 1)

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V, int e) {
        return a.C % V == 0 && vector_rows(a.x, V, e) && at16(a.y) && at16(a.init) && at16(a.final_state);
    };
    CONV_DISPATCH(conv_fwd_t, vec)
}

hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V, int e) {
        return a.C % V == 0 && vector_rows(a.x, V, e) && at16(a.y) && at16(a.init) && at16(a.final_state);
    };
    CONV_DISPATCH(conv_step_t, vec)
}

hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V, int e) {
        return a.C % V == 0 && vector_rows(a.x, V, e) && vector_rows(a.dy, V, e) && at16(a.dx) && at16(a.init) &&
               at16(a.dfinal) && at16(a.dinit);
    };
    CONV_DISPATCH(conv_bwd_t, vec)
}

}  // namespace ssd
