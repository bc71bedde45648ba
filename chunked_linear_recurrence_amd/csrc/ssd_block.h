// Arguments and launch functions of the operators around a scan: the short causal
// convolution, the selective scan with a decay per channel and state, and layer norm.
#pragma once

#include "libssdscan.h"
#include "ssd_common.h"

namespace ssd {

// A tensor [batch, seqlen, channels] whose channels are contiguous: token t of batch row b
// starts at p + b * bs + t * ts (elements).
struct View {
    const void *p;
    int64_t bs, ts;
};

template <typename T>
__device__ __forceinline__ const T *row_of(const View &v, int64_t b, int64_t t) {
    return reinterpret_cast<const T *>(v.p) + b * v.bs + t * v.ts;
}

// A launch holds fewer than 2^32 threads along a dimension.  A call of several launches checks
// all of them before the first.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

struct ConvArgs {
    int64_t batch;
    int L, C, W, dtype;
    uint32_t flags;
    View x;
    const float *w, *bias;        // [C, W]; [C] or null
    const void *init;             // [batch, W-1, C] or null
    const int32_t *lengths;       // [batch] or null
    void *y, *final_state;        // forward: [batch, L, C]; [batch, W-1, C] or null
    // backward
    View dy;
    const void *dfinal;           // [batch, W-1, C] or null
    void *dx, *dinit;             // [batch, L, C]; [batch, W-1, C] or null
    float *dw, *dbias;            // [C, W]; [C] or null
    float *part;                  // workspace: [conv_bwd_rows, W+1, C] partial sums
};

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t s);
int64_t conv_bwd_rows(int64_t batch, int64_t L, int64_t C, int32_t dtype);
bool conv_supported(int W);

struct NormArgs {
    int64_t rows;
    int D, dtype;
    const void *x;
    int64_t x_stride;             // elements between rows of x
    const float *w, *bias;        // [D] or null
    float eps;
    void *y;                      // [rows, D]
    float *mean, *rstd;           // [rows]; forward: written when not null
    // backward
    const void *dy;
    int64_t dy_stride;
    void *dx;                     // [rows, D]
    float *dw, *db;               // [D] or null
    float *part;                  // workspace: [norm_bwd_blocks, 2, D]
};

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t s);
int64_t norm_bwd_blocks(int64_t rows);

// Tokens between two kept states of the selective scan.
constexpr int kKeep = 8;

struct SelArgs {
    int64_t batch;
    int L, D, N, G, dtype;
    uint32_t flags;
    View u, delta, z, B, C;       // z.p may be null; B and C rows hold [G, N]
    const float *A;               // [D, N]
    const float *Dskip, *bias;    // [D] or null
    const float *init;            // [batch, D, N] or null
    const int32_t *lengths;       // [batch] or null
    void *y;                      // [batch, L, D]
    float *final_state;           // [batch, D, N] or null
    float *keep;                  // kept states or null (where each lies: sel_keep_slot)
    int tiles;                    // tiles of 64 channels per group
    int nc, T;                    // chunks and tokens per chunk (T a multiple of kKeep)
    float *S;                     // workspace [batch, nc, G*tiles, N, 64]
    float *sumdt;                 // workspace [batch, nc, G*tiles, 64]
    // backward
    View dy;
    const float *dfinal;
    void *du, *ddelta, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dinit;
    float *part_bc;               // [sel_bwd_parts, batch, L, G, 2, N]: dB, dC partial sums
    float *part_par;              // [batch, nc, G*tiles, N + 2, 64]: dA, dD, dbias partial sums
};

inline int sel_tiles(int64_t D, int64_t G) { return (int)((D / G + 63) / 64); }

bool sel_supported(int64_t N);
// Tiles of 64 channels that one workgroup of the backward takes (its 4 waves are tiles times
// blocks of 16 states), and workgroups per group of channels.
inline int sel_bwd_tiles(int64_t N) { return (int)(64 / N); }
inline int sel_bwd_parts(int64_t D, int64_t G, int64_t N) {
    return (sel_tiles(D, G) + sel_bwd_tiles(N) - 1) / sel_bwd_tiles(N);
}
// Chunks of the sequence: *nc chunks of *T tokens (at least 16) so that about cut.target waves
// run, for `waves` waves per chunk; one chunk, and so a single pass, from cut.enough waves on
// and up to cut.single tokens.
struct SelCut {
    int64_t target, enough, single;
};
void sel_chunks(int64_t waves, const SelCut &cut, int64_t L, int *nc, int *T);
hipError_t launch_sel_fwd(const SelArgs &a, hipStream_t s);
hipError_t launch_sel_bwd(const SelArgs &a, hipStream_t s);
hipError_t launch_sel_pass(const SelArgs &a, bool reverse, hipStream_t s);
hipError_t launch_sel_local_reverse(const SelArgs &a, hipStream_t s);

struct SelStepArgs {
    int64_t batch;
    int D, N, G, dtype;
    uint32_t flags;
    const void *u, *delta, *z, *B, *C;
    int64_t u_bs, delta_bs, z_bs, B_bs, C_bs;
    const float *A, *Dskip, *bias, *state_in;
    float *state_out;
    void *y;
};
hipError_t launch_sel_step(const SelStepArgs &a, hipStream_t s);

// ---------------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------------
constexpr float kLog2eF = 1.44269504088896340736f;
constexpr float kLn2F = 0.69314718055994530942f;

// V consecutive elements as one access (V * sizeof(T) bytes, naturally aligned).
template <typename T, int V>
struct Pack {
    typedef __attribute__((ext_vector_type(V))) T type;
};
template <typename T>
struct Pack<T, 1> {
    typedef T type;
};

template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::type load_pack(const T *p) {
    return *reinterpret_cast<const typename Pack<T, V>::type *>(p);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Pack<T, V>::type &q, float (&v)[V]) {
    if constexpr (V == 1) v[0] = to_f32(q);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)q[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_f32(T *p, const float (&v)[V]) {
    typename Pack<T, V>::type q;
    if constexpr (V == 1) q = from_f32<T>(v[0]);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = from_f32<T>(v[i]);
    }
    *reinterpret_cast<typename Pack<T, V>::type *>(p) = q;
}

__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }   // ~1 ulp

// 1 / (1 + e^-v): e^-v overflows to infinity for v below -88 and the quotient is then 0.
__device__ __forceinline__ float sigmoid_f32(float v) { return rcp_fast(1.f + exp2_fast(-v * kLog2eF)); }

__device__ __forceinline__ float silu_f32(float v) { return v * sigmoid_f32(v); }

// d/dv (v sigmoid(v))
__device__ __forceinline__ float dsilu_f32(float v) {
    const float s = sigmoid_f32(v);
    return s * fmaf(v, 1.f - s, 1.f);
}

// log(1 + e^v) and, in *sig, its derivative.  With w = fl(1 + e^v) the logarithm of w misses
// what the addition rounded off; (e^v - (w - 1)) / w puts it back, so small results keep
// their relative accuracy.  Above 20 the result is v to float32.  NaN stays NaN.
__device__ __forceinline__ float softplus_f32(float v, float *sig) {
    const float e = exp2_fast(v * kLog2eF), w = 1.f + e, r = rcp_fast(w);
    const float l = fmaf(__builtin_amdgcn_logf(w), kLn2F, (e - (w - 1.f)) * r);
    *sig = v > 20.f ? 1.f : e * r;
    return v > 20.f ? v : l;
}

// The same in base 2: log2(1 + 2^v) without its derivative and without a division.  What the
// addition rounded off is at most 2^-24 where w < 2, where it is added undivided (1/w > 1/2
// changes it by less than its own rounding of the logarithm's terms); where w is larger, that
// bound is below the result's own rounding.  From 126 on the result is v.
__device__ __forceinline__ float softplus2_f32(float v) {
    const float e = exp2_fast(v), w = 1.f + e;
    const float c = __builtin_amdgcn_fmed3f(e - (w - 1.f), -0x1p-24f, 0x1p-24f);
    return v > 126.f ? v : fmaf(c, kLog2eF, __builtin_amdgcn_logf(w));
}

// Sum over `rows` values a stride apart, for the 64 columns of a workgroup of W waves (p: this
// lane's column).  Each wave adds a contiguous share in order, 8 loads in flight at a time, and
// the first wave adds the shares in order; its lanes receive the result.
template <int W>
__device__ __forceinline__ float rows_sum(const float *p, int64_t rows, int64_t stride, float (&red)[W][64]) {
    const int lane = threadIdx.x % 64, k = threadIdx.x / 64;
    const int64_t end = rows * (k + 1) / W;
    float s = 0.f;
    for (int64_t r = rows * k / W; r < end; r += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[min(r + i, end - 1) * stride];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += r + i < end ? v[i] : 0.f;
    }
    red[k][lane] = s;
    __syncthreads();
    s = 0.f;
    if (k == 0)
#pragma unroll
        for (int w = 0; w < W; ++w) s += red[w][lane];
    return s;
}

__device__ __forceinline__ int row_length(const int32_t *lengths, int64_t b, int L) {
    if (!lengths) return L;
    return max(0, min(lengths[b], L));
}

}  // namespace ssd
