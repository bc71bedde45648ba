// Device code shared by the selective scan's forward and backward kernels.
//
// A tile is 64 channels of one group, one lane each; a lane keeps its channel's N states in
// registers.  B_t and C_t are the same for all lanes, so they are read through the scalar
// cache into scalar registers, which the vector units take as operands directly.
#pragma once

#include "ssd_block.h"

namespace ssd {

// N consecutive activations at a wave-uniform address (4-byte aligned), in scalar registers.
template <typename T, int N>
struct Uniform;
typedef const __attribute__((address_space(4))) uint32_t *scalar_ptr;

template <int N>
struct Uniform<float, N> {
    uint32_t w[N];
    __device__ __forceinline__ void load(const float *p) {
        scalar_ptr s = (scalar_ptr)(uintptr_t)p;
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = s[i];
    }
    __device__ __forceinline__ float operator[](int i) const { return __builtin_bit_cast(float, w[i]); }
};
template <int N>
struct Uniform<bf16, N> {
    uint32_t w[N / 2];
    __device__ __forceinline__ void load(const bf16 *p) {
        scalar_ptr s = (scalar_ptr)(uintptr_t)p;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = s[i];
    }
    __device__ __forceinline__ float operator[](int i) const {
        return __builtin_bit_cast(float, (i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    }
};

// Coefficients (rows of B or C) fetched together, one batch while the last is used.  A use of
// scalar loads waits for all that are in flight, so a batch cannot run further ahead than one;
// in bfloat16 it holds 32 states: 2 tokens of 16, or one token of 32, or half of one of 64
// (float32 batches of 16 states take as many scalar registers).
template <typename T, int N>
struct Batch {
    static constexpr int kBlocks = sizeof(T) == 2 ? 2 : 1;            // of 16 states
    static constexpr int kTokens = N == 16 ? kBlocks : 1;
    Uniform<T, 16> u[kBlocks];
    // row(k): the address of token k's coefficients; the batch that starts at token k, state n0
    template <typename F>
    __device__ __forceinline__ void load(F row, int k, int n0) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) u[i].load(kTokens > 1 ? row(k + i) : row(k) + n0 + 16 * i);
    }
};

// The same value, unknown to the compiler: addresses of unrolled tokens are then formed where
// they are used instead of all at once, which the scalar registers cannot hold.
__device__ __forceinline__ int hidden(int v) {
    asm volatile("" : "+s"(v));
    return v;
}
template <typename I>
__device__ __forceinline__ I hidden_lane(I v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ float masked(float v, uint32_t bits) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & bits);
}

// Keeps a running sum where it is written: the compiler otherwise moves a chain of additions
// whose result is used late past the branches in between, and holds all the terms until then.
__device__ __forceinline__ void pinned(float &v) { asm volatile("" : "+v"(v)); }

// A wave's tile: group, the lane's channel and its place in the [D] tensors.
struct SelTile {
    int tt, g;
    uint32_t d;
    bool live;
};

// Element d of a row.  The row's address is the same for all lanes and kept apart from the
// lane's offset, so that the load or store takes a scalar base and one 32-bit vector offset
// that serves all tensors, with no 64-bit vector arithmetic.
template <typename T>
using Global = __attribute__((address_space(1))) T;
template <typename T>
__device__ __forceinline__ Global<T> *lane_address(T *row, uint32_t d) {
    uint64_t a = (uint64_t)row;
    asm volatile("" : "+s"(a));
    return (Global<T> *)((Global<char> *)a + d * (uint32_t)sizeof(T));
}
// The rows of one batch row of a view: token t at p + t * ts bytes (the host has checked that
// ts fits), two scalar multiplications and two additions.
template <typename T>
struct Rows {
    const char *p;
    uint32_t ts;
    __device__ __forceinline__ Rows(const View &v, int64_t b)
        : p(reinterpret_cast<const char *>(v.p) + b * v.bs * (int64_t)sizeof(T)), ts((uint32_t)(v.ts * (int64_t)sizeof(T))) {}
    __device__ __forceinline__ const T *at(int t) const {
        return reinterpret_cast<const T *>(p + (uint64_t)(uint32_t)t * ts);
    }
};
template <typename T>
__device__ __forceinline__ T lane_load(const T *row, uint32_t d) {
    return *lane_address(row, d);
}
template <typename T>
__device__ __forceinline__ void lane_store(T *row, uint32_t d, T v) {
    *lane_address(row, d) = v;
}
__device__ __forceinline__ SelTile sel_tile(const SelArgs &a, int tt) {
    SelTile q;
    const int per = a.D / a.G;
    q.tt = tt;
    q.g = tt / a.tiles;
    const int c = (tt % a.tiles) * 64 + (int)(threadIdx.x % 64);
    q.live = c < per;
    q.d = (uint32_t)(q.g * per + min(c, per - 1));       // idle lanes read a channel that exists
    return q;
}

template <int N>
__device__ __forceinline__ void sel_rates(const SelArgs &a, uint32_t d, int n0, float scale, float (&A)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) A[n] = a.A[(int64_t)d * a.N + n0 + n] * scale;
}

// The step size of one token in base 2 (dt log2(e), so that its decays are 2^(dt2 A)), from
// delta and the bias times log2(e).  Chosen without a branch, which would cut the unrolled
// tokens into blocks that cannot be scheduled together.
__device__ __forceinline__ float sel_dt2(float delta, float bias2, bool softplus) {
    const float v = fmaf(delta, kLog2eF, bias2), l = softplus2_f32(v);
    return softplus ? l : v;
}
// The step size itself, and its derivative by delta.
__device__ __forceinline__ float sel_dt(float raw, bool softplus, float *sig) {
    float s;
    const float dt = softplus_f32(raw, &s);
    *sig = softplus ? s : 1.f;
    return softplus ? dt : raw;
}

// Offset of chunk c of batch row b in S (floats), lane included; state n is at n * 64.
__device__ __forceinline__ int64_t sel_slot(const SelArgs &a, int64_t b, int c, int tt, int width) {
    return (((b * a.nc + c) * (a.G * a.tiles) + tt) * (int64_t)width) * 64 + threadIdx.x % 64;
}
__device__ __forceinline__ int64_t sel_keep_slot(const SelArgs &a, int64_t b, int sub, int tt, int n0) {
    const int64_t nsub = (a.L + kKeep - 1) / kKeep;
    return (((b * nsub + sub) * (a.G * a.tiles) + tt) * (int64_t)a.N + n0) * 64 + threadIdx.x % 64;
}

}  // namespace ssd
