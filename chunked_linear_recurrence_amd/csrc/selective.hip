// Selective scan with a decay of its own for every channel d and state n:
//
//     dt_t = softplus(delta_t + bias)   (or delta_t + bias)
//     h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t u_t B_t[n]
//     y_t = sum_n C_t[n] h_t[n] + D u_t;   out_t = y_t z_t sigmoid(z_t)   (or y_t)
//
// The decays differ for every (channel, state), so the products do not factor into matrix
// products as they do with one decay per head: the work is, per (token, channel, state), an
// exponential (two issue slots), two multiplications and two fused multiply-adds on the vector
// units, against 4 activations moved per (token, channel).  A tile of 64 channels and 16 states
// takes 96 slots of 4 cycles a token for that, 128 with step sizes, gate and conversions; the
// counters show the vector units busy for all of (1)'s time and over 80% of (3)'s.  So memory
// does not bound the scan (2 TB/s at 32768 tokens of 2048 channels: 177-194 us in (1), 232-259 in
// (3); 312 and 411 with 32 states, 648 and 933 with 64), and each slot counts: the step size is
// kept in base 2, so that a decay is one multiplication and one 2^x; B and C are scalar operands;
// addresses are scalar; everything that would sit
// between a load and its use is fetched 3 tokens early.  The float32 matrix instructions that
// could form dt u B for 16 states at once were measured not to overlap with vector work on the
// same SIMD, and bfloat16 ones would round the state.
//
// Chunks.  A tile of 64 channels is one wave, and few channels at batch 1 leave the GPU
// empty, so the sequence is cut into chunks: (1) every chunk's end state from a zero state,
// and the sum of its dt; (2) the states passed from chunk to chunk,
// h <- exp(A sum dt) h + S; (3) every chunk again from the state that enters it.  (1) and (2)
// are skipped where there are waves enough without.
#include <type_traits>

#include "ssd_sel.h"

namespace ssd {

constexpr int kSelWaves = 4;     // independent waves per workgroup
constexpr int kAhead = 3, kRing = 4;   // steps that activations are fetched ahead, and their places

// Wave -> (batch row, chunk, tile); tiles are neighbours, so the waves of a workgroup share
// B and C.  False past the last unit.
__device__ __forceinline__ bool sel_unit(const SelArgs &a, int nchunks, int64_t *b, int *c, int *tt) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int ntt = a.G * a.tiles;
    const int64_t u = (int64_t)blockIdx.x * kSelWaves + wave;
    if (u >= a.batch * nchunks * ntt) return false;
    *tt = (int)(u % ntt);
    *c = (int)(u / ntt % nchunks);
    *b = u / ntt / nchunks;
    return true;
}

// (1), and its mirror for the backward (REV): the carry a_t g_t that leaves the chunk's first
// token when none enters at its end, g_t = C_t r_t + a_{t+1} g_{t+1}.
// GATE (with REV): z is given.
template <typename T, int N, bool REV, bool GATE>
__global__ __launch_bounds__(256) void sel_local_kernel(SelArgs a) {
    int64_t b;
    int c, tt;
    if (!sel_unit(a, a.nc - 1, &b, &c, &tt)) return;
    if (REV) ++c;
    const SelTile q = sel_tile(a, tt);
    const int len = row_length(a.lengths, b, a.L);
    const int begin = c * a.T, end = min(begin + a.T, len);
    const bool softplus = (a.flags & SSD_FLAG_SOFTPLUS) != 0;
    const float bias2 = a.bias ? a.bias[q.d] * kLog2eF : 0.f;
    float A[N], h[N], sum = 0.f;
    sel_rates<N>(a, q.d, 0, 1.f, A);
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.f;
    const Rows<T> coef(REV ? a.C : a.B, b), val(REV ? a.dy : a.u, b), delta(a.delta, b), zr(a.z, b);
    // Step k is token begin + k, or end - 1 - k backwards.  Activations are fetched kAhead steps
    // early into a ring, coefficients one batch early.
    T dv[kRing], xv[kRing], zv[kRing];
    auto token = [&](int k) { return hidden(REV ? end - 1 - min(k, end - begin - 1) : begin + min(k, end - begin - 1)); };
    uint32_t d = q.d;
    auto fetch = [&](int k, int slot) {
        const int t = token(k);
        dv[slot] = lane_load(delta.at(t), d);
        xv[slot] = lane_load(val.at(t), d);
        if (GATE) zv[slot] = lane_load(zr.at(t), d);
    };
    typedef Batch<T, N> Coef;
    Coef cf, cn;
    auto row = [&](int k) { return coef.at(token(k)) + q.g * N; };
    if (begin < end) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(k, k);
        cn.load(row, 0, 0);
    }
    auto step = [&](int k, int slot) {
        const float dt2 = sel_dt2(to_f32(dv[slot]), bias2, softplus);
        sum += dt2;
        float x = to_f32(xv[slot]);
        if (!REV) x = dt2 * (x * kLn2F);
        else if (GATE) x *= silu_f32(to_f32(zv[slot]));
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 16) {
            const int u = Coef::kTokens > 1 ? slot % Coef::kTokens : n0 / 16 % Coef::kBlocks;
            if (u == 0) {
                cf = cn;
                if (n0 + 16 * Coef::kBlocks < N) cn.load(row, k, n0 + 16 * Coef::kBlocks);
                else cn.load(row, k + Coef::kTokens, 0);
            }
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                const float e = exp2_fast(dt2 * A[n0 + n]), c = cf.u[u][n];
                h[n0 + n] = REV ? e * fmaf(x, c, h[n0 + n]) : fmaf(e, h[n0 + n], x * c);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    const int steps = max(end - begin, 0);
    int k0 = 0;
    for (; k0 + kRing <= steps; k0 += kRing) {
        d = hidden_lane(d);      // known to be 32 bits here: a scalar base and a vector offset, no 64-bit sum
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            fetch(k0 + i + kAhead, (i + kAhead) % kRing);
            step(k0 + i, i);
        }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (k0 + i < steps) step(k0 + i, i);
    float *S = a.S + sel_slot(a, b, c, tt, N);
#pragma unroll
    for (int n = 0; n < N; ++n) S[n * 64] = h[n];
    a.sumdt[sel_slot(a, b, c, tt, 1)] = sum;
}

// (2).  A workgroup takes one state of one tile: its W waves share out the chunks, each first
// joins its own (decay and end state), the joined parts meet in LDS, and each then walks its
// chunks from the state that enters them.  Each chunk's slot of S receives the state (REV: the
// carry) that enters it.  W is such that a wave has at most 16 chunks, whose values it then
// holds in registers; it waits for memory once.
constexpr int kPassChunks = 16;

// 2^x h + s, x the exponent of many tokens' decays together.  Where rates are positive 2^x may be
// beyond float32 although every token's decay and every state is within it.  BIG: some lane's x is
// above 127, and 2^x is taken as two finite factors: a state of zero stays zero, and another
// overflows only where the result does.
template <bool BIG>
__device__ __forceinline__ float joined(float x, float h, float s) {
    if (!BIG) return fmaf(exp2_fast(x), h, s);
    const bool big = x > 127.f;
    const float e = exp2_fast(big ? 127.f : x), more = exp2_fast(big ? fminf(x - 127.f, 127.f) : 0.f);
    return fmaf(e, more * h, s);
}

template <bool REV, int W>
__global__ __launch_bounds__(64 * W) void sel_pass_kernel(SelArgs a) {
    constexpr int U = kPassChunks;
    __shared__ float part[W][2][64];
    const int ntt = a.G * a.tiles, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int n = blockIdx.x % a.N, tt = blockIdx.x / a.N % ntt;
    const int64_t b = blockIdx.x / a.N / ntt;
    const SelTile q = sel_tile(a, tt);
    const float A = a.A[(int64_t)q.d * a.N + n];
    const float *first = REV ? a.dfinal : a.init;
    const int64_t cs = (int64_t)ntt * a.N * 64, ds = (int64_t)ntt * 64;
    float *S = a.S + ((b * a.nc * ntt + tt) * (int64_t)a.N + n) * 64 + lane;
    const float *sd = a.sumdt + (b * a.nc * ntt + tt) * (int64_t)64 + lane;
    // in walking order, the last chunk has no values of its own (none follows it)
    const int c0 = (int)((int64_t)a.nc * wave / W), c1 = (int)((int64_t)a.nc * (wave + 1) / W);
    auto slot = [&](int c) { return (int64_t)(REV ? a.nc - 1 - c : c); };
    float h = 0.f, total = 0.f, s[U], d[U];
    auto walk = [&](bool write) {
        for (int c = c0; c < c1; c += U) {
            if (!write || c1 - c0 > U || W == 1) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int64_t at = slot(min(min(c + i, c1 - 1), a.nc - 2));
                    s[i] = S[at * cs];
                    d[i] = sd[at * ds];
                }
            }
            const float again = hidden_lane(A);      // the products are formed where they are used, not held
            bool big = false;
#pragma unroll
            for (int i = 0; i < U; ++i) big |= again * d[i] > 127.f;
            auto steps = [&](auto any_big) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (c + i < c1) {
                        if (write) S[slot(c + i) * cs] = h;
                        h = joined<any_big()>(A * d[i], h, s[i]);
                        total += d[i];
                    }
                }
            };
            if (__any(big)) steps(std::true_type());
            else steps(std::false_type());
        }
    };
    if (W > 1) {
        walk(false);
        part[wave][0][lane] = h;
        part[wave][1][lane] = total;
        __syncthreads();
    }
    h = first ? first[(b * a.D + q.d) * (int64_t)a.N + n] : 0.f;
    for (int w = 0; w < wave; ++w) h = joined<true>(A * part[w][1][lane], h, part[w][0][lane]);
    walk(true);
}

// (3); GATE: z is given
template <typename T, int N, bool GATE>
__global__ __launch_bounds__(256) void sel_scan_kernel(SelArgs a) {
    int64_t b;
    int c, tt;
    if (!sel_unit(a, a.nc, &b, &c, &tt)) return;
    const SelTile q = sel_tile(a, tt);
    const int len = row_length(a.lengths, b, a.L);
    const int begin = c * a.T, stop = min(begin + a.T, a.L), end = min(stop, len);
    const bool softplus = (a.flags & SSD_FLAG_SOFTPLUS) != 0;
    const float bias2 = a.bias ? a.bias[q.d] * kLog2eF : 0.f, skip = a.Dskip ? a.Dskip[q.d] : 0.f;
    float A[N], h[N];
    sel_rates<N>(a, q.d, 0, 1.f, A);
    const float *S = a.S + sel_slot(a, b, c, tt, N);
    const float *h0 = a.init ? a.init + (b * a.D + q.d) * (int64_t)N : nullptr;
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = a.nc > 1 ? S[n * 64] : (h0 ? h0[n] : 0.f);
    T *y = reinterpret_cast<T *>(a.y) + b * a.L * (int64_t)a.D;
    const Rows<T> delta(a.delta, b), u(a.u, b), z(a.z, b), B(a.B, b), C(a.C, b);
    T dv[kRing], uv[kRing], zv[kRing];
    auto token = [&](int t) { return hidden(min(t, end - 1)); };
    uint32_t d = q.d;
    auto fetch = [&](int k, int slot) {
        const int t = token(k);
        dv[slot] = lane_load(delta.at(t), d);
        uv[slot] = lane_load(u.at(t), d);
        if (GATE) zv[slot] = lane_load(z.at(t), d);
    };
    typedef Batch<T, N> Coef;
    Coef Bt, Ct, Bn, Cn;
    auto coefficients = [&](int k, int n0) {
        Bn.load([&](int t) { return B.at(token(t)) + q.g * N; }, k, n0);
        Cn.load([&](int t) { return C.at(token(t)) + q.g * N; }, k, n0);
    };
    if (begin < end) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(begin + k, k);
        coefficients(begin, 0);
    }
    auto step = [&](int t, int slot) {
        const float dt2 = sel_dt2(to_f32(dv[slot]), bias2, softplus);
        const float ut = to_f32(uv[slot]), x = dt2 * (ut * kLn2F);
        float acc[2] = {skip * ut, 0.f};
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 16) {
            const int u = Coef::kTokens > 1 ? slot % Coef::kTokens : n0 / 16 % Coef::kBlocks;
            if (u == 0) {
                Bt = Bn;
                Ct = Cn;
                if (n0 + 16 * Coef::kBlocks < N) coefficients(t, n0 + 16 * Coef::kBlocks);
                else coefficients(t + Coef::kTokens, 0);
            }
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                h[n0 + n] = fmaf(exp2_fast(dt2 * A[n0 + n]), h[n0 + n], x * Bt.u[u][n]);
                acc[n & 1] = fmaf(Ct.u[u][n], h[n0 + n], acc[n & 1]);
            }
        }
        float o = acc[0] + acc[1];
        if (GATE) o *= silu_f32(to_f32(zv[slot]));
        lane_store(y + t * (int64_t)a.D, d, from_f32<T>(o));      // an idle lane: the same value in the same place
        __builtin_amdgcn_sched_barrier(0);
    };
    auto keep_state = [&](int t) {
        if (a.keep && t % kKeep == 0) {
            float *kp = a.keep + sel_keep_slot(a, b, t / kKeep, tt, 0);
#pragma unroll
            for (int n = 0; n < N; ++n) kp[n * 64] = h[n];
        }
    };
    static_assert(kKeep % kRing == 0, "states are kept between groups of kRing tokens");
    int t0 = begin;
    for (; t0 + kRing <= end; t0 += kRing) {
        d = hidden_lane(d);
        keep_state(t0);
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            fetch(t0 + i + kAhead, (i + kAhead) % kRing);
            step(t0 + i, i);
        }
    }
    if (t0 < end) keep_state(t0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (t0 + i < end) step(t0 + i, i);
    if (q.live) {
        for (int t = max(begin, end); t < stop; ++t) lane_store(y + t * (int64_t)a.D, q.d, from_f32<T>(0.f));
        if (a.final_state && c == a.nc - 1) {
            float *f = a.final_state + (b * a.D + q.d) * (int64_t)N;
#pragma unroll
            for (int n = 0; n < N; ++n) f[n] = h[n];
        }
    }
}

// One token.  The state, 8 bytes read and written per element, is the traffic: N/4 threads
// share a channel, each with 4 states (one 16-byte access each way), and add their parts of
// the sum over n with wave shuffles.  256 streams of 2048 channels: 16 us for 71 MB.
template <typename T, int N>
__global__ __launch_bounds__(256) void sel_step_kernel(SelStepArgs a) {
    constexpr int Q = N / 4;
    const int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) / Q;
    const int n0 = threadIdx.x % Q * 4;
    if (k >= a.batch * a.D) return;                     // whole channels leave together
    const int64_t b = k / a.D;
    const int d = (int)(k % a.D), g = d / (a.D / a.G);
    const bool softplus = (a.flags & SSD_FLAG_SOFTPLUS) != 0;
    const T *Bp = reinterpret_cast<const T *>(a.B) + b * a.B_bs + g * N + n0;
    const T *Cp = reinterpret_cast<const T *>(a.C) + b * a.C_bs + g * N + n0;
    const float *A = a.A + (int64_t)d * N + n0;
    const f32x4 s = *reinterpret_cast<const f32x4 *>(a.state_in + k * N + n0);
    const float u = to_f32(reinterpret_cast<const T *>(a.u)[b * a.u_bs + d]);
    const float dt2 = sel_dt2(to_f32(reinterpret_cast<const T *>(a.delta)[b * a.delta_bs + d]),
                              a.bias ? a.bias[d] * kLog2eF : 0.f, softplus);
    const float x = dt2 * (u * kLn2F);
    f32x4 h;
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(exp2_fast(dt2 * A[i]), s[i], x * to_f32(Bp[i]));
        part = fmaf(to_f32(Cp[i]), h[i], part);
    }
    *reinterpret_cast<f32x4 *>(a.state_out + k * N + n0) = h;
#pragma unroll
    for (int o = Q / 2; o >= 1; o >>= 1) part += __shfl_xor(part, o, 64);
    if (n0 == 0) {
        float o = fmaf(a.Dskip ? a.Dskip[d] : 0.f, u, part);
        if (a.z) o *= silu_f32(to_f32(reinterpret_cast<const T *>(a.z)[b * a.z_bs + d]));
        reinterpret_cast<T *>(a.y)[k] = from_f32<T>(o);
    }
}

bool sel_supported(int64_t N) { return N == 16 || N == 32 || N == 64; }

void sel_chunks(int64_t waves, const SelCut &cut, int64_t L, int *nc, int *T) {
    const int64_t n = waves >= cut.enough || L <= cut.single ? 1 : (cut.target + waves - 1) / waves;
    int64_t t = (L + n - 1) / n;
    t = (t + kKeep - 1) / kKeep * kKeep;
    if (t < 16) t = 16;
    *nc = (int)((L + t - 1) / t);
    *T = (int)t;
}

static hipError_t sel_grid(int64_t units, uint32_t *blocks) {
    const int64_t n = (units + kSelWaves - 1) / kSelWaves;
    if (n < 1 || !grid_fits(n, 64 * kSelWaves)) return hipErrorInvalidValue;
    *blocks = (uint32_t)n;
    return hipSuccess;
}

// Several chunks are cut only where a chunk has fewer than 2048 waves, so the grids of (1) and (2)
// are far below a launch's limit.
hipError_t launch_sel_pass(const SelArgs &a, bool reverse, hipStream_t s) {
    const int64_t n = a.batch * a.G * a.tiles * a.N;
#define SEL_PASS(W)                                                                        \
    do {                                                                                   \
        if (reverse) sel_pass_kernel<true, W><<<(uint32_t)n, 64 * W, 0, s>>>(a);           \
        else sel_pass_kernel<false, W><<<(uint32_t)n, 64 * W, 0, s>>>(a);                  \
    } while (0)
    if (a.nc <= kPassChunks) SEL_PASS(1);
    else if (a.nc <= 4 * kPassChunks) SEL_PASS(4);
    else if (a.nc <= 8 * kPassChunks) SEL_PASS(8);
    else SEL_PASS(16);
#undef SEL_PASS
    return hipGetLastError();
}

template <typename T, int N>
static hipError_t sel_fwd_t(const SelArgs &a, hipStream_t s) {
    const int64_t per = a.batch * a.G * a.tiles;
    uint32_t blocks;
    hipError_t e;
    if (a.nc > 1) {
        if ((e = sel_grid(per * (a.nc - 1), &blocks)) != hipSuccess) return e;
        sel_local_kernel<T, N, false, false><<<blocks, 256, 0, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if ((e = launch_sel_pass(a, false, s)) != hipSuccess) return e;
    }
    if ((e = sel_grid(per * a.nc, &blocks)) != hipSuccess) return e;
    if (a.z.p) sel_scan_kernel<T, N, true><<<blocks, 256, 0, s>>>(a);
    else sel_scan_kernel<T, N, false><<<blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int N>
static hipError_t sel_step_t(const SelStepArgs &a, hipStream_t s) {
    const int64_t n = (a.batch * a.D * (N / 4) + 255) / 256;
    if (!grid_fits(n, 256)) return hipErrorInvalidValue;
    sel_step_kernel<T, N><<<(uint32_t)n, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int N>
static hipError_t sel_rev_t(const SelArgs &a, hipStream_t s) {
    uint32_t blocks;
    hipError_t e = sel_grid(a.batch * a.G * a.tiles * (a.nc - 1), &blocks);
    if (e != hipSuccess) return e;
    if (a.z.p) sel_local_kernel<T, N, true, true><<<blocks, 256, 0, s>>>(a);
    else sel_local_kernel<T, N, true, false><<<blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

#define SEL_PICK(FN, T)                          \
    switch (a.N) {                               \
        case 16: return FN<T, 16>(a, s);         \
        case 32: return FN<T, 32>(a, s);         \
        case 64: return FN<T, 64>(a, s);         \
        default: return hipErrorInvalidValue;    \
    }
#define SEL_DISPATCH(FN)                         \
    if (a.dtype == 1) { SEL_PICK(FN, bf16) }     \
    SEL_PICK(FN, float)

hipError_t launch_sel_fwd(const SelArgs &a, hipStream_t s) { SEL_DISPATCH(sel_fwd_t) }
hipError_t launch_sel_step(const SelStepArgs &a, hipStream_t s) { SEL_DISPATCH(sel_step_t) }
hipError_t launch_sel_local_reverse(const SelArgs &a, hipStream_t s) { SEL_DISPATCH(sel_rev_t) }

}  // namespace ssd
