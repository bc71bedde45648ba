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
// tokens per TS that the caches hold; the loads of 8 tokens (4 in the backward) are started
// together, as a store in between may touch what a later load reads as far as the compiler
// knows.  8 x 4096 tokens of 2048 channels in bfloat16: 59 us, 4.6 TB/s (a copy of the same
// size reaches 4.8).  Backward, the same size and 4 taps: 112 us, 3.6 TB/s; with 8 channels a
// thread it takes 236 registers, so two waves a SIMD have too few loads on their way.
#include "ssd_block.h"

namespace ssd {

constexpr int kConvWaves = 4;       // token segments per workgroup, one wave each
constexpr int kConvFwdTokens = 16, kConvBwdTokens = 32;   // tokens per wave at most

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
__device__ __forceinline__ void conv_input(const ConvArgs &a, const ConvUnit &q, int t, int len, float (&v)[V]) {
    typename Pack<T, V>::type p = {};
    if (t >= 0 && t < len) p = load_pack<T, V>(row_of<T>(a.x, q.b, t) + q.c);
    else if (t < 0 && a.init)
        p = load_pack<T, V>(reinterpret_cast<const T *>(a.init) + (q.b * (W - 1) + (t + W - 1)) * a.C + q.c);
    unpack<T, V>(p, v);
}

// Row k of a state [batch, W-1, C].
template <typename T, int W>
__device__ __forceinline__ T *conv_state(void *p, const ConvArgs &a, const ConvUnit &q, int k) {
    return reinterpret_cast<T *>(p) + (q.b * (W - 1) + k) * a.C + q.c;
}

template <int W, int V>
__device__ __forceinline__ void conv_weights(const ConvArgs &a, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.w[(int64_t)min(c + i, a.C - 1) * W + j];
        bias[i] = a.bias ? a.bias[min(c + i, a.C - 1)] : 0.f;
    }
}

constexpr int kConvLoads = 8;       // tokens whose loads are in flight together

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int TS) {
    constexpr int U = kConvLoads;
    const ConvUnit q = conv_unit<V>(a.L, a.C, TS);
    if (q.c >= a.C || q.t0 >= a.L) return;
    const int len = row_length(a.lengths, q.b, a.L);
    const bool silu = (a.flags & SSD_FLAG_SILU) != 0;
    float w[W][V], bias[V], win[W][V];
    conv_weights<W, V>(a, q.c, w, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q, q.t0 - (W - 1) + k, len, win[k]);
    // The state of the row's last token: the thread that holds the row's start writes it, as
    // it alone reads the incoming state, which may be the same memory.
    if (q.t0 == 0 && a.final_state) {
        float f[W - 1][V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q, len - (W - 1) + k, len, f[k]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_f32<T, V>(conv_state<T, W>(a.final_state, a, q, k), f[k]);
    }
    const int t1 = min(q.t0 + TS, a.L), end = min(t1, len);
    T *y = reinterpret_cast<T *>(a.y) + (q.b * a.L + q.t0) * (int64_t)a.C + q.c;
    int t = q.t0;
    while (t < end) {
        typename Pack<T, V>::type p[U];
#pragma unroll
        for (int i = 0; i < U; ++i) p[i] = load_pack<T, V>(row_of<T>(a.x, q.b, min(t + i, end - 1)) + q.c);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (t < end) {
                float o[V];
                unpack<T, V>(p[k], win[W - 1]);
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
                store_f32<T, V>(y, o);
                y += a.C;
                ++t;
            }
        }
    }
    const float zero[V] = {};
    for (; t < t1; ++t, y += a.C) store_f32<T, V>(y, zero);
}

// One token: y from the state and x, and the state moved on by one (in place or not).  Its few
// kilobytes are latency alone (2.4 us at 1536 channels): one access a thread, one wave a workgroup.
template <typename T, int W, int V>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvArgs a) {
    const int nt = (a.C + V - 1) / V;
    const int64_t k = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (k >= a.batch * nt) return;
    const ConvUnit q = {k / nt, 0, (int)(k % nt) * V};
    float w[W][V], bias[V], win[W][V], o[V];
    conv_weights<W, V>(a, q.c, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) conv_input<T, W, V>(a, q, j - (W - 1), 1, win[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float s = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[j][i], win[j][i], s);
        o[i] = (a.flags & SSD_FLAG_SILU) ? silu_f32(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_f32<T, V>(conv_state<T, W>(a.final_state, a, q, j), win[j + 1]);
    store_f32<T, V>(reinterpret_cast<T *>(a.y) + q.b * a.C + q.c, o);
}

// Backward.  A wave of tokens [t0, t1) recomputes pre and dpre for [t0, t1 + W-1) and writes
// dx for its own tokens (the wave at the row's start also the W-1 positions of the carried
// state); dw and dbias are summed over its own tokens only.  The sums of the workgroup's
// waves meet in LDS and leave as one row of partial sums.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_bwd_rows_of(const ConvArgs &a, const ConvUnit &q, int TS, float (&dw)[W][V],
                                                 float (&db)[V]) {
    constexpr int U = 4;
    const int len = row_length(a.lengths, q.b, a.L);
    const bool silu = (a.flags & SSD_FLAG_SILU) != 0;
    float w[W][V], bias[V], win[W][V], dp[W][V];       // dp[j] = dpre of token s - j
    conv_weights<W, V>(a, q.c, w, bias);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<T, W, V>(a, q, q.t0 - (W - 1) + k, len, win[k]);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dp[j][i] = 0.f;
    const int t1 = min(q.t0 + TS, a.L), stop = t1 + W - 1;
    const int first = q.t0 == 0 ? -(W - 1) : q.t0;
    for (int s0 = q.t0; s0 < stop; s0 += U) {
        typename Pack<T, V>::type px[U] = {}, pg[U] = {};
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int t = min(s0 + k, min(len, stop) - 1);
            if (t >= s0) {
                px[k] = load_pack<T, V>(row_of<T>(a.x, q.b, t) + q.c);
                pg[k] = load_pack<T, V>(row_of<T>(a.dy, q.b, t) + q.c);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int s = s0 + k;
            if (s >= stop) break;
#pragma unroll
            for (int j = W - 1; j > 0; --j)
#pragma unroll
                for (int i = 0; i < V; ++i) dp[j][i] = dp[j - 1][i];
            if (s < len) {
                float g[V];
                unpack<T, V>(px[k], win[W - 1]);
                unpack<T, V>(pg[k], g);
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
            if (t >= first) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[i] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) o[i] = fmaf(w[j][i], dp[j][i], o[i]);
                }
                const int f = t - (len - (W - 1));         // this input's place in the final state
                if (a.dfinal && f >= 0 && f < W - 1) {
                    float g[V];
                    unpack<T, V>(load_pack<T, V>(conv_state<T, W>(const_cast<void *>(a.dfinal), a, q, f)), g);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] += g[i];
                }
                if (t >= 0)
                    store_f32<T, V>(reinterpret_cast<T *>(a.dx) + (q.b * a.L + t) * (int64_t)a.C + q.c, o);
                else if (a.dinit) store_f32<T, V>(conv_state<T, W>(a.dinit, a, q, t + W - 1), o);
            }
        }
    }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int TS) {
    __shared__ float red[kConvWaves - 1][(W + 1) * V][64];
    const ConvUnit q = conv_unit<V>(a.L, a.C, TS);
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (q.c < a.C && q.t0 < a.L) conv_bwd_rows_of<T, W, V>(a, q, TS, dw, db);
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

// Tokens per wave: `most`, halved while fewer than 4 waves run on each of the 1024 SIMDs, to 4
// at least (W-1 tokens per wave are read, and in the backward computed, twice).
static int conv_tokens(int64_t batch, int64_t L, int64_t C, int32_t dtype, int most) {
    const int vec = dtype == 1 ? 8 : 4, V = C % vec == 0 ? vec : 1;
    const int64_t tiles = batch * ((C + 64 * V - 1) / (64 * V));
    int ts = most;
    while (ts > 4 && tiles * ((L + ts - 1) / ts) < 4096) ts /= 2;
    return ts;
}
static int conv_bwd_tokens(int64_t batch, int64_t L, int64_t C, int32_t dtype) {
    return conv_tokens(batch, L, C, dtype, kConvBwdTokens);
}

int64_t conv_bwd_rows(int64_t batch, int64_t L, int64_t C, int32_t dtype) {
    const int64_t per = kConvWaves * conv_bwd_tokens(batch, L, C, dtype);
    return batch * ((L + per - 1) / per);
}

template <typename T, int W, int V>
static hipError_t conv_fwd_t(const ConvArgs &a, hipStream_t s) {
    const int TS = conv_tokens(a.batch, a.L, a.C, a.dtype, kConvFwdTokens);
    const int64_t nct = (a.C + 64 * V - 1) / (64 * V), ntb = (a.L + kConvWaves * TS - 1) / (kConvWaves * TS);
    const int64_t n = a.batch * ntb * nct;
    if (!grid_fits(n, 256)) return hipErrorInvalidValue;
    conv_fwd_kernel<T, W, V><<<(uint32_t)n, 256, 0, s>>>(a, TS);
    return hipGetLastError();
}

template <typename T, int W, int V>
static hipError_t conv_step_t(const ConvArgs &a, hipStream_t s) {
    const int64_t n = (a.batch * ((a.C + V - 1) / V) + 63) / 64;
    if (!grid_fits(n, 64)) return hipErrorInvalidValue;
    conv_step_kernel<T, W, V><<<(uint32_t)n, 64, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int W, int V>
static hipError_t conv_bwd_t(const ConvArgs &a, hipStream_t s) {
    const int64_t nct = (a.C + 64 * V - 1) / (64 * V), rows = conv_bwd_rows(a.batch, a.L, a.C, a.dtype);
    const int64_t sums = ((int64_t)(W + 1) * a.C + 63) / 64;
    if (!grid_fits(rows * nct, 256) || !grid_fits(sums, 1024)) return hipErrorInvalidValue;
    conv_bwd_kernel<T, W, V><<<(uint32_t)(rows * nct), 256, 0, s>>>(a, conv_bwd_tokens(a.batch, a.L, a.C, a.dtype));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    conv_bwd_sum_kernel<<<(uint32_t)sums, 1024, 0, s>>>(a.part, rows, a.C, W, a.dw, a.dbias);
    return hipGetLastError();
}

// 16-byte accesses need every tensor's start, and every row's, on a 16-byte boundary; other
// tensors are taken channel by channel.
static bool vector_rows(const View &v, int V) { return ((uintptr_t)v.p & 15u) == 0 && v.bs % V == 0 && v.ts % V == 0; }
static bool at16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

#define CONV_PICK(FN, T, V)                          \
    switch (a.W) {                                   \
        case 2: return FN<T, 2, V>(a, s);            \
        case 3: return FN<T, 3, V>(a, s);            \
        case 4: return FN<T, 4, V>(a, s);            \
        default: return hipErrorInvalidValue;        \
    }
#define CONV_DISPATCH(FN, VEC)                       \
    if (a.dtype == 1) {                              \
        if (VEC(8)) { CONV_PICK(FN, bf16, 8) }       \
        CONV_PICK(FN, bf16, 1)                       \
    }                                                \
    if (VEC(4)) { CONV_PICK(FN, float, 4) }          \
    CONV_PICK(FN, float, 1)

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V) {
        return a.C % V == 0 && vector_rows(a.x, V) && at16(a.y) && at16(a.init) && at16(a.final_state);
    };
    CONV_DISPATCH(conv_fwd_t, vec)
}

hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V) {
        return a.C % V == 0 && vector_rows(a.x, V) && at16(a.y) && at16(a.init) && at16(a.final_state);
    };
    CONV_DISPATCH(conv_step_t, vec)
}

hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t s) {
    auto vec = [&](int V) {
        return a.C % V == 0 && vector_rows(a.x, V) && vector_rows(a.dy, V) && at16(a.dx) && at16(a.init) &&
               at16(a.dfinal) && at16(a.dinit);
    };
    CONV_DISPATCH(conv_bwd_t, vec)
}

}  // namespace ssd
