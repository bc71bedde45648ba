// The norms after and before a block with its gate, its scale and the residual, and their
// backward.  Each row of D channels, rms(v) = v / sqrt(mean(v^2) + eps):
//
//     t = branch silu(gate);   p = rms(t) post;   s = residual + scale p;   y = rms(s) pre
//
//     ds = dtotal + rs (g - shat mean(g shat)),  g = dy pre, shat = s rs
//     dp = ds scale;   dt = rt (h - that mean(h that)),  h = dp post, that = t rt
//     dresidual = ds;  dbranch = dt silu(gate);  dgate = dt branch silu'(gate)
//     dpre = sum over rows of dy shat;  dscale = of ds p;  dpost = of dp that
//
// What is not given drops out.  A stream of up to 5 elements in the forward and 8 in the
// backward per channel; a row is read once and held in registers between its sums (1, 4 or 8
// waves, the fewest that hold it; rows wider than that, or narrower than 16 bytes and off them,
// are read again for each sum).  s is
// formed again in the backward in float32, from the same reads that its rounded copy would
// cost, so no rounding of s enters a gradient.  The three column sums are kept in registers
// over a workgroup's rows, leave it as one row of partial sums, and a second kernel adds those
// in order, so results do not depend on scheduling.  Bound by memory: 32768 x 2048 in bfloat16 with
// everything given 131 us forward (5.1 TB/s) and 208 + 6 backward (5.2 TB/s).
#include "residual_norm.h"

namespace ssd {

constexpr int kRnFwdBlocks = 1024, kRnBwdBlocks = 512;   // workgroups at most

template <int WPR> constexpr int rn_threads() { return WPR == 8 ? 512 : 256; }
// Whether registers hold the next row beside the backward's current one
template <typename T, int V, int K> constexpr bool rn_ahead() { return K * V * (int)sizeof(T) / 4 <= 8; }
// Whether the backward's parameters are set to 1 where another thread counts, or its sums over a row leave
// those values out: 8 waves of bfloat16 have no registers left (4000 x 7001 290 us, 224 with the sums; 1
// wave, 20000 x 777, 77 and 82, 4 waves, 8000 x 3001, 155 and 165; float32 by 8, 3000 x 8001, 401 and 443)
template <typename T, int WPR> constexpr bool rn_own() { return sizeof(T) == 4 || WPR < 8; }
template <int WPR> constexpr int rn_rows() { return WPR == 1 ? 4 : 1; }       // rows a workgroup holds at a time

// Where a thread's k-th access of V values to a row of D begins.  ANY: rows may start anywhere and end
// inside an access, which then begins V values before the row's end; the first `over` of its
// values are another thread's, read as zeros and not stored.  (Loads of single values for the
// row's end made the workgroup wait for one wave: 16000 rows of 2047 channels in bfloat16, 255 us
// backward.)
template <int V, int WPR, bool ANY>
struct Place {
    int c, over;
    bool on;
    __device__ __forceinline__ Place(int k, int tid, int D) {
        const int at = (k * 64 * WPR + tid) * V;
        on = at < D;
        c = ANY ? min(at, D - V) : at;
        over = ANY ? at - c : 0;
    }
};
template <typename T, int V, int WPR, bool ANY>
__device__ __forceinline__ void store_at(void *p, int64_t row, int D, const Place<V, WPR, ANY> &at, const float (&v)[V]) {
    T *y = reinterpret_cast<T *>(p) + row * D + at.c;
    if constexpr (!ANY) {
        store_f32<T, V>(y, v);
    } else if (at.over == 0) {
        typename Pack<T, V>::type q;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = from_f32<T>(v[i]);
        __builtin_memcpy(y, &q, sizeof(q));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= at.over) y[i] = from_f32<T>(v[i]);
    }
}

template <typename T, int V, int K, int WPR, bool ANY>
struct RowRegs {
    typename Pack<T, V>::type v[K];
    // this thread's accesses of a row (null: none); those past the row are left alone
    __device__ __forceinline__ void load(const T *x, int D, int tid) {
        if (!x) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Place<V, WPR, ANY> at(k, tid, D);
            if (at.on) __builtin_memcpy(&v[k], x + at.c, sizeof(v[k]));
        }
    }
    // of what was loaded, another thread's values to zeros (apart, so that loads may be on their way)
    __device__ __forceinline__ void own(int D, int tid) {
        if constexpr (ANY) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Place<V, WPR, ANY> at(k, tid, D);
                if (at.on && at.over > 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i < at.over) v[k][i] = from_f32<T>(0.f);
                }
            }
        }
    }
};

__device__ __forceinline__ float gate_f32(float z) { return silu_limit(z, sigmoid_f32(z)); }

template <typename T>
__device__ __forceinline__ const T *row_at(const void *p, int64_t row, int64_t stride) {
    return p ? reinterpret_cast<const T *>(p) + row * stride : nullptr;
}

// A parameter's values, 1 where it is not given.  WHOLE: in whole accesses also off 16 bytes.
template <int V, int K, int WPR, bool ANY, bool WHOLE>
__device__ __forceinline__ void load_params(const float *p, int D, int tid, float (&v)[K][V]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Place<V, WPR, ANY> at(k, tid, D);
        if constexpr (ANY && WHOLE) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = 1.f;
            if (p && at.on) __builtin_memcpy(v[k], p + at.c, sizeof(v[k]));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = p && at.on ? p[at.c + i] : 1.f;
        }
    }
}
// Of what was loaded, another thread's values to 1: 0 x 1 in the row's sums, not 0 x infinity.  By
// selects in the forward (4000 x 7001 62 us, 69 in a branch), in a branch that only a row's last
// thread takes in the backward (20000 x 777 77 us, 87 by selects).
template <int V, int K, int WPR, bool ANY, bool BRANCH>
__device__ __forceinline__ void own_params(int D, int tid, float (&v)[K][V]) {
    if constexpr (ANY) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Place<V, WPR, ANY> at(k, tid, D);
            if (BRANCH && at.over <= 0) continue;
            if (BRANCH) asm volatile("");
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = i < at.over ? 1.f : v[k][i];
        }
    }
}

// dot and the products x y of an access, but the first `over`
template <int V, bool SOME>
__device__ __forceinline__ float add_own(int over, const float (&x)[V], const float (&y)[V], float dot) {
    if (!SOME || over == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) dot = fmaf(x[i], y[i], dot);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i >= over) dot = fmaf(x[i], y[i], dot);
    }
    return dot;
}

template <typename T, int V, int K, int WPR, bool ANY>
__global__ __launch_bounds__(rn_threads<WPR>()) void residual_norm_fwd_kernel(ResidualNormArgs a) {
    __shared__ float red[16];
    constexpr int R = rn_rows<WPR>();
    const int tid = WPR == 1 ? threadIdx.x % 64 : threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * R + (WPR == 1 ? threadIdx.x / 64 : 0), by = (int64_t)gridDim.x * R;
    float post[K][V], scale[K][V], pre[K][V];
    load_params<V, K, WPR, ANY, true>(a.post, a.D, tid, post);
    load_params<V, K, WPR, ANY, true>(a.scale, a.D, tid, scale);
    load_params<V, K, WPR, ANY, true>(a.pre, a.D, tid, pre);
    own_params<V, K, WPR, ANY, false>(a.D, tid, post);
    own_params<V, K, WPR, ANY, false>(a.D, tid, scale);
    own_params<V, K, WPR, ANY, false>(a.D, tid, pre);
    RowRegs<T, V, K, WPR, ANY> bn = {}, zn = {}, rn = {};
    auto fetch = [&](int64_t row) {
        bn.load(row_at<T>(a.branch, row, a.branch_stride), a.D, tid);
        zn.load(row_at<T>(a.gate, row, a.gate_stride), a.D, tid);
        rn.load(row_at<T>(a.residual, row, a.residual_stride), a.D, tid);
    };
    if (first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += by) {
        RowRegs<T, V, K, WPR, ANY> b = bn, z = zn, r = rn;
        if (row + by < a.rows) fetch(row + by);
        b.own(a.D, tid);
        if (a.gate) z.own(a.D, tid);                             // 0 x infinity
        if (a.residual) r.own(a.D, tid);
        float v[K][V];
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            unpack<T, V>(b.v[k], v[k]);
            if (a.gate) {
                float g[V];
                unpack<T, V>(z.v[k], g);
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] *= gate_f32(g[i]);
            }
            if (Place<V, WPR, ANY>(k, tid, a.D).on)
#pragma unroll
                for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
        }
        float rt = 1.f;
        if (a.post) rt = 1.f / sqrtf(row_sum<WPR>(sq, red) / a.D + a.eps);
        sq = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float res[V];
            unpack<T, V>(r.v[k], res);
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = fmaf(v[k][i] * rt * post[k][i], scale[k][i], a.residual ? res[i] : 0.f);
            const Place<V, WPR, ANY> at(k, tid, a.D);
            if (at.on) {
                store_at<T, V, WPR, ANY>(a.total, row, a.D, at, v[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
            }
        }
        float rs = 1.f;
        if (a.pre) {
            rs = 1.f / sqrtf(row_sum<WPR>(sq, red) / a.D + a.eps);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Place<V, WPR, ANY> at(k, tid, a.D);
                if (at.on) {
#pragma unroll
                    for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rs * pre[k][i];
                    store_at<T, V, WPR, ANY>(a.y, row, a.D, at, v[k]);
                }
            }
        }
        if (a.stats && tid == 0) {
            a.stats[row] = rt;
            a.stats[a.rows + row] = rs;
        }
    }
}

// Rows that registers do not hold: one workgroup a row, from row `first` of a launch on, a pass over it
// for each sum and one to store.  Bound by accesses of single elements: 2000 x 16384 in bfloat16 260 us
// forward and 726 backward (1.3 and 0.7 TB/s; 415 and 1028 by workgroups that loop over rows), and narrow
// rows by 1024 threads for each: 4.2 M x 3 23.5 and 47.6 ms.
template <typename T>
struct WideRow {
    const T *b, *z, *r;
    const ResidualNormArgs &a;
    __device__ __forceinline__ WideRow(const ResidualNormArgs &args, int64_t row)
        : b(row_at<T>(args.branch, row, args.branch_stride)), z(row_at<T>(args.gate, row, args.gate_stride)),
          r(row_at<T>(args.residual, row, args.residual_stride)), a(args) {}
    __device__ __forceinline__ float t(int c) const { return z ? to_f32(b[c]) * gate_f32(to_f32(z[c])) : to_f32(b[c]); }
    __device__ __forceinline__ float p(float t, float rt, int c) const { return a.post ? t * rt * a.post[c] : t; }
    __device__ __forceinline__ float s(float p, int c) const {
        return fmaf(p, a.scale ? a.scale[c] : 1.f, r ? to_f32(r[c]) : 0.f);
    }
};

template <typename T>
__global__ __launch_bounds__(1024) void residual_norm_fwd_wide_kernel(ResidualNormArgs a, int64_t first) {
    __shared__ float red[16];
    const int64_t row = first + blockIdx.x;
    const WideRow<T> w(a, row);
    float rt = 1.f, rs = 1.f, sq = 0.f;
    if (a.post) {
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            const float t = w.t(c);
            sq = fmaf(t, t, sq);
        }
        rt = 1.f / sqrtf(row_sum<16>(sq, red) / a.D + a.eps);
    }
    if (a.pre) {
        sq = 0.f;
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            const float s = w.s(w.p(w.t(c), rt, c), c);
            sq = fmaf(s, s, sq);
        }
        rs = 1.f / sqrtf(row_sum<16>(sq, red) / a.D + a.eps);
    }
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float s = w.s(w.p(w.t(c), rt, c), c);      // before the store: total may be residual
        reinterpret_cast<T *>(a.total)[row * a.D + c] = from_f32<T>(s);
        if (a.pre) reinterpret_cast<T *>(a.y)[row * a.D + c] = from_f32<T>(s * rs * a.pre[c]);
    }
    if (a.stats && threadIdx.x == 0) {
        a.stats[row] = rt;
        a.stats[a.rows + row] = rs;
    }
}

template <typename T, int V, int K, int WPR, bool ANY>
__global__ __launch_bounds__(rn_threads<WPR>()) void residual_norm_bwd_kernel(ResidualNormArgs a) {
    __shared__ float red[16];
    __shared__ float cols[WPR == 1 ? 3 * 64 * V * K : 1];
    constexpr int R = rn_rows<WPR>();
    constexpr bool OWN = rn_own<T, WPR>();
    const int wave = threadIdx.x / 64, tid = WPR == 1 ? threadIdx.x % 64 : threadIdx.x;
    const int64_t first = (int64_t)blockIdx.x * R + (WPR == 1 ? wave : 0), by = (int64_t)gridDim.x * R;
    float post[K][V], scale[K][V], pre[K][V], sums[3][K][V];
    load_params<V, K, WPR, ANY, OWN>(a.post, a.D, tid, post);
    load_params<V, K, WPR, ANY, OWN>(a.scale, a.D, tid, scale);
    load_params<V, K, WPR, ANY, OWN>(a.pre, a.D, tid, pre);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) sums[q][k][i] = 0.f;
    RowRegs<T, V, K, WPR, ANY> bn = {}, zn = {}, rn = {}, yn = {}, tn = {};
    float rt_n = 1.f, rs_n = 1.f;
    auto fetch = [&](int64_t row) {
        bn.load(row_at<T>(a.branch, row, a.branch_stride), a.D, tid);
        zn.load(row_at<T>(a.gate, row, a.gate_stride), a.D, tid);
        yn.load(row_at<T>(a.dy, row, a.dy_stride), a.D, tid);
        if (a.dy) rn.load(row_at<T>(a.residual, row, a.residual_stride), a.D, tid);     // s is needed for its norm alone
        tn.load(row_at<T>(a.dtotal, row, a.dtotal_stride), a.D, tid);
        rt_n = a.stats[row];
        rs_n = a.stats[a.rows + row];
    };
    if (first < a.rows) fetch(first);
    if constexpr (OWN) {
        own_params<V, K, WPR, ANY, true>(a.D, tid, post);
        own_params<V, K, WPR, ANY, true>(a.D, tid, scale);
        own_params<V, K, WPR, ANY, true>(a.D, tid, pre);
    }
    for (int64_t row = first; row < a.rows; row += by) {
        RowRegs<T, V, K, WPR, ANY> bq = bn, zq = zn, rq = rn, yq = yn, tq = tn;
        const float rt = rt_n, rs = rs_n;
        if (rn_ahead<T, V, K>() && row + by < a.rows) fetch(row + by);
        bq.own(a.D, tid);
        if (a.dy) yq.own(a.D, tid);
        if (a.dtotal) tq.own(a.D, tid);
        float that[K][V], d[K][V], s[K][V];
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            unpack<T, V>(bq.v[k], that[k]);
            if (a.gate) {
                float z[V];
                unpack<T, V>(zq.v[k], z);
#pragma unroll
                for (int i = 0; i < V; ++i) that[k][i] *= gate_f32(z[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) that[k][i] *= rt;
            unpack<T, V>(tq.v[k], d[k]);                       // zeros where dtotal is not given
            if (a.dy) {
                float r[V], dy[V];
                unpack<T, V>(rq.v[k], r);
                unpack<T, V>(yq.v[k], dy);
                const Place<V, WPR, ANY> at(k, tid, a.D);
                float g[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[k][i] = fmaf(that[k][i] * post[k][i], scale[k][i], r[i]) * rs;      // shat
                    g[i] = dy[i] * pre[k][i];
                    if (at.on) sums[0][k][i] = fmaf(dy[i], s[k][i], sums[0][k][i]);
                }
                if (at.on) dot = add_own<V, ANY && !OWN>(at.over, g, s[k], dot);
            }
        }
        if (a.dy) {
            dot = row_sum<WPR>(dot, red) / a.D;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dy[V];
                unpack<T, V>(yq.v[k], dy);
#pragma unroll
                for (int i = 0; i < V; ++i) d[k][i] = fmaf(rs, dy[i] * pre[k][i] - s[k][i] * dot, d[k][i]);
            }
        }
        dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Place<V, WPR, ANY> at(k, tid, a.D);
            if (at.on) {
                if (a.dresidual) store_at<T, V, WPR, ANY>(a.dresidual, row, a.D, at, d[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sums[1][k][i] = fmaf(d[k][i], that[k][i] * post[k][i], sums[1][k][i]);
                    d[k][i] *= scale[k][i];                    // dp
                    sums[2][k][i] = fmaf(d[k][i], that[k][i], sums[2][k][i]);
                    d[k][i] *= post[k][i];
                }
                dot = add_own<V, ANY && !OWN>(at.over, d[k], that[k], dot);
            }
        }
        if (a.post) {
            dot = row_sum<WPR>(dot, red) / a.D;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) d[k][i] = rt * (d[k][i] - that[k][i] * dot);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Place<V, WPR, ANY> at(k, tid, a.D);
            if (!at.on) continue;
            if (a.gate) {
                float z[V], b[V], dz[V];
                unpack<T, V>(zq.v[k], z);
                unpack<T, V>(bq.v[k], b);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float sg = sigmoid_f32(z[i]);
                    dz[i] = d[k][i] * b[i] * sg * dsilu_limit(z[i], sg);
                    d[k][i] *= silu_limit(z[i], sg);
                }
                store_at<T, V, WPR, ANY>(a.dgate, row, a.D, at, dz);
            }
            store_at<T, V, WPR, ANY>(a.dbranch, row, a.D, at, d[k]);
        }
        if (!rn_ahead<T, V, K>() && row + by < a.rows) fetch(row + by);
    }
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * 3 * a.D;
    if constexpr (WPR == 1) {
        // the 4 waves add their sums in wave order
        constexpr int M = 64 * V * K;
        for (int w = 0; w < 4; ++w) {
            if (wave == w) {
#pragma unroll
                for (int q = 0; q < 3; ++q)
#pragma unroll
                    for (int k = 0; k < K; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float &at = cols[q * M + (k * V + i) * 64 + tid];      // lanes side by side
                            at = (w ? at : 0.f) + sums[q][k][i];
                        }
            }
            __syncthreads();
        }
        for (int m = threadIdx.x; m < 3 * M; m += 256) {
            const int q = m / M, l = m % 64, k = m % M / 64 / V, i = m / 64 % V;
            const Place<V, WPR, ANY> at(k, l, a.D);
            if (at.on && i >= at.over) part[(int64_t)q * a.D + at.c + i] = cols[m];
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Place<V, WPR, ANY> at(k, tid, a.D);
            if (at.on)
#pragma unroll
                for (int q = 0; q < 3; ++q)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i >= at.over) part[(int64_t)q * a.D + at.c + i] = sums[q][k][i];
        }
    }
}

// Rows that registers do not hold: the same sums by passes over the row; the terms of the three
// column sums are left to the kernel below, which needs each row's two means (rows of `mean`).
template <typename T>
__device__ __forceinline__ void wide_terms(const ResidualNormArgs &a, const WideRow<T> &w, int64_t row, int c, float rt,
                                           float rs, float mean_s, float &that, float &p, float &shat, float &dy, float &ds) {
    that = w.t(c) * rt;
    p = a.post ? that * a.post[c] : that;
    ds = a.dtotal ? to_f32(row_at<T>(a.dtotal, row, a.dtotal_stride)[c]) : 0.f;
    shat = dy = 0.f;
    if (a.dy) {
        shat = w.s(p, c) * rs;
        dy = to_f32(row_at<T>(a.dy, row, a.dy_stride)[c]);
        ds = fmaf(rs, dy * a.pre[c] - shat * mean_s, ds);
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void residual_norm_bwd_wide_kernel(ResidualNormArgs a, int64_t first) {
    __shared__ float red[16];
    const int64_t row = first + blockIdx.x;
    const WideRow<T> w(a, row);
    const float rt = a.stats[row], rs = a.stats[a.rows + row];
    float that, p, shat, dy, ds, mean_s = 0.f, mean_t = 0.f, dot = 0.f;
    if (a.dy) {
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            wide_terms(a, w, row, c, rt, rs, 0.f, that, p, shat, dy, ds);
            dot = fmaf(dy * a.pre[c], shat, dot);
        }
        mean_s = row_sum<16>(dot, red) / a.D;
    }
    if (a.post) {
        dot = 0.f;
        for (int c = threadIdx.x; c < a.D; c += 1024) {
            wide_terms(a, w, row, c, rt, rs, mean_s, that, p, shat, dy, ds);
            dot = fmaf(ds * (a.scale ? a.scale[c] : 1.f) * a.post[c], that, dot);
        }
        mean_t = row_sum<16>(dot, red) / a.D;
    }
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        wide_terms(a, w, row, c, rt, rs, mean_s, that, p, shat, dy, ds);
        if (a.dresidual) reinterpret_cast<T *>(a.dresidual)[row * a.D + c] = from_f32<T>(ds);
        float d = ds * (a.scale ? a.scale[c] : 1.f);
        if (a.post) d = rt * (d * a.post[c] - that * mean_t);
        if (a.gate) {
            const float z = to_f32(w.z[c]), sg = sigmoid_f32(z);
            reinterpret_cast<T *>(a.dgate)[row * a.D + c] = from_f32<T>(d * to_f32(w.b[c]) * sg * dsilu_limit(z, sg));
            d *= silu_limit(z, sg);
        }
        reinterpret_cast<T *>(a.dbranch)[row * a.D + c] = from_f32<T>(d);
    }
    if (threadIdx.x == 0) a.mean[row] = mean_s;
}

template <typename T>
__global__ __launch_bounds__(256) void residual_norm_bwd_cols_kernel(ResidualNormArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D) return;
    float sums[3] = {0.f, 0.f, 0.f};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const WideRow<T> w(a, row);
        float that, p, shat, dy, ds;
        wide_terms(a, w, row, c, a.stats[row], a.stats[a.rows + row], a.mean[row], that, p, shat, dy, ds);
        sums[0] = fmaf(dy, shat, sums[0]);
        sums[1] = fmaf(ds, p, sums[1]);
        sums[2] = fmaf(ds * (a.scale ? a.scale[c] : 1.f), that, sums[2]);
    }
    float *part = a.part + (int64_t)blockIdx.y * 3 * a.D + c;
#pragma unroll
    for (int q = 0; q < 3; ++q) part[(int64_t)q * a.D] = sums[q];
}

__global__ __launch_bounds__(1024) void residual_norm_sum_kernel(ResidualNormArgs a, int rows) {
    __shared__ float red[16][64];
    const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x % 64, cols = 3 * (int64_t)a.D;
    const float s = rows_sum<16>(a.part + min(col, cols - 1), rows, cols, red);
    if (threadIdx.x >= 64 || col >= cols) return;
    float *out = col < a.D ? a.dpre : col < 2 * (int64_t)a.D ? a.dscale : a.dpost;
    if (out) out[col % a.D] = s;
}

// Channels that registers hold: from one access of 16 bytes on
constexpr int kRnMost = 8192;
static bool rn_held(int64_t D, int dtype) { return D >= (dtype == 1 ? 8 : 4) && D <= kRnMost; }
constexpr int64_t kRnWideRows = (1 << 22) - 1;           // other rows of one launch: below 2^32 threads

int64_t residual_norm_bwd_blocks(int64_t rows) { return rows < kRnBwdBlocks ? rows : kRnBwdBlocks; }
size_t residual_norm_mean_rows(int64_t rows, int64_t D, int dtype) { return rn_held(D, dtype) ? 0 : (size_t)rows; }

static bool rn_sums(const ResidualNormArgs &a) { return a.dpre || a.dscale || a.dpost; }

// Every row that the call reads or writes starts on 16 bytes and is a whole number of them.
static bool rn_vec(const ResidualNormArgs &a) {
    const int64_t e = a.dtype == 1 ? 2 : 4;
    auto at = [&](const void *p, int64_t stride) { return ((uintptr_t)p & 15u) == 0 && (!p || stride * e % 16 == 0); };
    return a.D * e % 16 == 0 && at(a.branch, a.branch_stride) && at(a.gate, a.gate_stride) &&
           at(a.residual, a.residual_stride) && at(a.dy, a.dy_stride) && at(a.dtotal, a.dtotal_stride) && at(a.y, a.D) &&
           at(a.total, a.D) && at(a.dbranch, a.D) && at(a.dgate, a.D) && at(a.dresidual, a.D);
}

bool residual_norm_fits(const ResidualNormArgs &a) {
    return rn_held(a.D, a.dtype) || grid_fits((3 * (int64_t)a.D + 63) / 64, 1024);
}

template <typename T, int V, int K, int WPR, bool ANY>
static hipError_t rn_fwd(const ResidualNormArgs &a, hipStream_t s) {
    constexpr int R = rn_rows<WPR>();
    const int64_t n = min((a.rows + R - 1) / R, (int64_t)kRnFwdBlocks);
    residual_norm_fwd_kernel<T, V, K, WPR, ANY><<<(uint32_t)n, rn_threads<WPR>(), 0, s>>>(a);
    return hipGetLastError();
}

static hipError_t rn_sum(const ResidualNormArgs &a, int64_t blocks, hipStream_t s) {
    if (!rn_sums(a)) return hipSuccess;
    residual_norm_sum_kernel<<<(uint32_t)((3 * (int64_t)a.D + 63) / 64), 1024, 0, s>>>(a, (int)blocks);
    return hipGetLastError();
}

template <typename T, int V, int K, int WPR, bool ANY>
static hipError_t rn_bwd(const ResidualNormArgs &a0, hipStream_t s) {
    constexpr int R = rn_rows<WPR>();
    ResidualNormArgs a = a0;
    if (!rn_sums(a)) a.part = nullptr;
    const int64_t n = min((a.rows + R - 1) / R, residual_norm_bwd_blocks(a.rows));
    residual_norm_bwd_kernel<T, V, K, WPR, ANY><<<(uint32_t)n, rn_threads<WPR>(), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : rn_sum(a, n, s);
}

template <typename K>
static hipError_t rn_wide(K kernel, const ResidualNormArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < a.rows && e == hipSuccess; first += kRnWideRows) {
        kernel<<<(uint32_t)min(a.rows - first, kRnWideRows), 1024, 0, s>>>(a, first);
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
static hipError_t rn_fwd_wide(const ResidualNormArgs &a, hipStream_t s) {
    return rn_wide(residual_norm_fwd_wide_kernel<T>, a, s);
}

template <typename T>
static hipError_t rn_bwd_wide(const ResidualNormArgs &a, hipStream_t s) {
    hipError_t e = rn_wide(residual_norm_bwd_wide_kernel<T>, a, s);
    if (e != hipSuccess || !rn_sums(a)) return e;
    const int64_t n = residual_norm_bwd_blocks(a.rows);
    residual_norm_bwd_cols_kernel<T><<<dim3((a.D + 255) / 256, (uint32_t)n), 256, 0, s>>>(a);
    e = hipGetLastError();
    return e != hipSuccess ? e : rn_sum(a, n, s);
}

// The fewest waves that hold a row of D channels, 16 bytes an access and 16 values a thread at most.
#define RN_BF16(DIR, ANY)                                                \
    do {                                                                 \
        if (a.D <= 512) return rn_##DIR<bf16, 8, 1, 1, ANY>(a, s);       \
        if (a.D <= 1024) return rn_##DIR<bf16, 8, 2, 1, ANY>(a, s);      \
        if (a.D <= 2048) return rn_##DIR<bf16, 8, 1, 4, ANY>(a, s);      \
        if (a.D <= 4096) return rn_##DIR<bf16, 8, 2, 4, ANY>(a, s);      \
        return rn_##DIR<bf16, 8, 2, 8, ANY>(a, s);                       \
    } while (0)
#define RN_F32(DIR, ANY)                                                 \
    do {                                                                 \
        if (a.D <= 256) return rn_##DIR<float, 4, 1, 1, ANY>(a, s);      \
        if (a.D <= 512) return rn_##DIR<float, 4, 2, 1, ANY>(a, s);      \
        if (a.D <= 1024) return rn_##DIR<float, 4, 1, 4, ANY>(a, s);     \
        if (a.D <= 2048) return rn_##DIR<float, 4, 2, 4, ANY>(a, s);     \
        if (a.D <= 4096) return rn_##DIR<float, 4, 4, 4, ANY>(a, s);     \
        return rn_##DIR<float, 4, 4, 8, ANY>(a, s);                      \
    } while (0)

#define RN_LAUNCH(DIR)                                              \
    do {                                                            \
        const bool vec = rn_vec(a);                                 \
        if (!rn_held(a.D, a.dtype)) {                               \
            if (a.dtype == 1) return rn_##DIR##_wide<bf16>(a, s);   \
            return rn_##DIR##_wide<float>(a, s);                    \
        }                                                           \
        if (a.dtype == 1) {                                         \
            if (vec) RN_BF16(DIR, false);                           \
            RN_BF16(DIR, true);                                     \
        }                                                           \
        if (vec) RN_F32(DIR, false);                                \
        RN_F32(DIR, true);                                          \
    } while (0)

hipError_t launch_residual_norm_fwd(const ResidualNormArgs &a, hipStream_t s) { RN_LAUNCH(fwd); }
hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, hipStream_t s) { RN_LAUNCH(bwd); }

}  // namespace ssd
