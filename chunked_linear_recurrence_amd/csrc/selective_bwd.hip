// Backward of the selective scan (its forward's formulas are in selective.hip).  With
// r_t = dout_t silu(z_t) and, from the last token to the first,
//
//     g_t[n] = C_t[n] r_t + a_{t+1}[n] g_{t+1}[n],   a_t = exp(dt_t A)
//
// the gradients are
//
//     q_t = sum_n g_t B_t;  w_t[n] = g_t a_t h_{t-1};  ddt_t = u_t q_t + sum_n A w_t
//     du_t = dt_t q_t + D r_t;  ddelta_t = ddt_t d(softplus);  dz_t = dout_t y_t d(silu)(z_t)
//     dA[n] = sum_t dt_t w_t;  dB_t[n] = sum_d g_t dt_t u_t;  dC_t[n] = sum_d r_t h_t
//     dD = sum_t r_t u_t;  dbias = sum_t ddelta_t;  dinit = a_0 g_0
//
// The forward leaves the state before every 8th token (8 bytes a (token, channel) at N = 16:
// as much as its four activations).  From the last group of 8 tokens to the first, a wave (64
// channels, one lane each, 16 states) runs the group forward from that state, with the 8 tokens'
// states in registers, and then backward through them.  h_{t-1} is never recovered by division,
// which would lose it where decays are small.  The decays are computed a second time on the way
// back: keeping them too would take 128 more registers and leave one wave per SIMD.
//
// The sums over channels (dC on the way forward, dB on the way back) go through LDS: every lane
// writes the 16 products of a token, and each lane then adds a quarter of a column, one token
// later, so that the reads are covered by arithmetic.  The 4 waves of a workgroup are 64/N tiles
// times N/16 blocks of states; their sums meet in LDS, and one partial sum per workgroup goes
// to memory, added up in order by a last kernel, so that results do not depend on scheduling.
//
// 340 vector instructions a (token, 64 channels, 16 states) bound it: 2 x 4096 tokens of 2048
// channels take 226 to 246 us on different machines, the vector units busy for 76% of them with
// two waves a SIMD (240 registers and none in memory; 34 to 98 scalars are held in lanes).
#include "ssd_sel.h"

namespace ssd {

constexpr int kSB = 16;                  // states per wave
// The reduction buffer of a wave: a row of 16 products (and 4 of padding) per lane, 16 rows
// per quarter of the lanes, quarters 16 banks apart, so that both the 16-byte writes along a
// row and the reads down a column are free of bank conflicts.
constexpr int kRow = 20, kQuarter = 16 * kRow + 16;

// Orders a wave's LDS operations in the program, where its lanes read what other lanes wrote: the
// wave issues them in order, and this keeps the compiler from moving one past another.  No
// instruction.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename T, int N, bool GATE>
__global__ __launch_bounds__(256, 2) void sel_bwd_kernel(SelArgs a) {
    constexpr int NB = N / kSB, TPB = 4 / NB, K = kKeep;
    __shared__ __align__(16) float red[4][4 * kQuarter];
    __shared__ float comb[4][K][2][64];
    // dt, u, d(softplus) and r lane by lane.  A tile's NB waves each write the same values; the
    // barriers around the end of a group keep its waves from writing the next group's before all
    // have read this one's.
    __shared__ float tok[TPB][K][4][64];
    // where a tile has several blocks of states, each block's part of y, q and sum A w
    __shared__ float cross[NB > 1 ? 4 : 1][NB > 1 ? K : 1][3][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int parts = (a.tiles + TPB - 1) / TPB;
    const int pg = blockIdx.x % (parts * a.G), g = pg / parts, part = pg % parts;
    const int64_t bc = blockIdx.x / (parts * a.G);
    const int c = (int)(bc % a.nc);
    const int64_t b = bc / a.nc;
    const int tile = part * TPB + wave / NB, nb = wave % NB, n0 = nb * kSB;
    const bool real = tile < a.tiles;                       // a wave past the group's tiles only takes part in barriers
    SelTile q = sel_tile(a, g * a.tiles + (real ? tile : a.tiles - 1));
    q.live = q.live && real;
    const int len = row_length(a.lengths, b, a.L);
    const int begin = c * a.T, stop = min(begin + a.T, a.L), end = min(stop, len);
    const bool softplus = (a.flags & SSD_FLAG_SOFTPLUS) != 0;
    const float bias = a.bias ? a.bias[q.d] : 0.f, skip = a.Dskip ? a.Dskip[q.d] : 0.f;
    float A2[kSB], carry[kSB], dA[kSB], dD = 0.f, dbias = 0.f;
    sel_rates<kSB>(a, q.d, n0, kLog2eF, A2);
    const float *S = a.S + sel_slot(a, b, c, q.tt, N) + n0 * 64;
    const float *f0 = a.dfinal ? a.dfinal + (b * a.D + q.d) * (int64_t)N + n0 : nullptr;
#pragma unroll
    for (int n = 0; n < kSB; ++n) {
        carry[n] = a.nc > 1 ? S[n * 64] : (f0 ? f0[n] : 0.f);
        dA[n] = 0.f;
    }
    const uint32_t d = q.d;
    const Rows<T> r_u(a.u, b), r_delta(a.delta, b), r_dy(a.dy, b), r_z(a.z, b), r_B(a.B, b), r_C(a.C, b);
    // row t of an output [batch, L, D]
    const int64_t out_first = b * a.L * (int64_t)a.D;
    auto out_row = [&](void *p, int t) { return reinterpret_cast<T *>(p) + out_first + (uint64_t)(uint32_t)t * (uint32_t)a.D; };
    // Reads of tok go by a lane index of their own, so that the values come back from LDS and
    // are not kept in registers from the way forward to the way back.
    const int back = hidden_lane(lane);
    float *mine = red[wave] + (lane / 16) * kQuarter + (lane % 16) * kRow;
    const float *column = red[wave] + (lane / 16) * kQuarter + lane % 16;
    // All ones, or zeros where a token or the lane's channel is a copy of another, whose values
    // must add nothing to any sum (by bits: a product with 0 would keep infinities and NaN).
    const uint32_t live = q.live ? ~0u : 0u;

    // dz and dD of a token, given its y without the skip term
    auto finish_z = [&](int t, float u, float r, float gz, float y) {
        dD = fmaf(r, u, dD);
        if (GATE && q.live && t < end) lane_store(out_row(a.dz, t), d, from_f32<T>(gz * fmaf(skip, u, y)));
    };
    // du and ddelta of a token, given q and sum A w (base-2 rates)
    auto finish_u = [&](int t, float dt, float u, float sig, float r, float qq, float dw) {
        const float dl = fmaf(dw, kLn2F, u * qq) * sig;
        if (q.live && t < end) {
            dbias += dl;
            lane_store(out_row(a.du, t), d, from_f32<T>(fmaf(dt, qq, skip * r)));
            lane_store(out_row(a.ddelta, t), d, from_f32<T>(dl));
        }
    };
    // r = dout silu(z) and dout d(silu)(z), masked
    auto upstream = [&](T dyv, T zv, uint32_t in, float *r, float *gz) {
        *r = masked(to_f32(dyv), in);
        *gz = 0.f;
        if (GATE) {
            const float z = masked(to_f32(zv), in), s = sigmoid_f32(z);
            *gz = *r * s * fmaf(z, 1.f - s, 1.f);
            *r *= z * s;
        }
    };

    // The lane's quarter of column lane % 16 of the products in the buffer.  Reads are started
    // before the next token's products are written (a wave's LDS operations run in order) and
    // added up after its arithmetic.
    float col[16];
    auto column_read = [&]() {
        wave_order();
#pragma unroll
        for (int k = 0; k < 16; ++k) col[k] = column[k * kRow];
        wave_order();
    };
    auto column_sum = [&]() {
        float s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = (col[k] + col[4 + k]) + (col[8 + k] + col[12 + k]);
        return (s[0] + s[1]) + (s[2] + s[3]);
    };
    auto kept_state = [&](int t0, float (&h)[kSB]) {
        const float *kp = a.keep + sel_keep_slot(a, b, t0 / K, q.tt, n0);
#pragma unroll
        for (int n = 0; n < kSB; ++n) h[n] = kp[n * 64];
    };

    float h0[kSB], hn[kSB];
    Uniform<T, kSB> Bt, Ct, Bn, Cn;
    T dv[3], uv[3], dyv[3], zv[3];                          // tokens i, i + 1 and i + 2 of a group, by i mod 3
    // A token past the row's last is a copy of an earlier one: `in` is 0 for it.
    auto fetch = [&](int t0, int i) {
        const int t = hidden(min(t0 + i, end - 1));
        dv[i % 3] = lane_load(r_delta.at(t), d);
        uv[i % 3] = lane_load(r_u.at(t), d);
        dyv[i % 3] = lane_load(r_dy.at(t), d);
        if (GATE) zv[i % 3] = lane_load(r_z.at(t), d);
    };
    auto coefficients = [&](int t0, int i, Uniform<T, kSB> &B, Uniform<T, kSB> &C) {
        const int t = hidden(min(t0 + i, end - 1));
        B.load(r_B.at(t) + g * N + n0);
        C.load(r_C.at(t) + g * N + n0);
    };
    const int last = begin + (max(end - begin, 1) - 1) / K * K;
    if (begin < end) {
        kept_state(last, hn);
        fetch(last, 0);
        fetch(last, 1);
    }
    for (int t0 = last; t0 >= begin && t0 < end; t0 -= K) {
        const int m = min(K, end - t0);
        float hs[K][kSB];
#pragma unroll
        for (int n = 0; n < kSB; ++n) h0[n] = hn[n];
        // Forward through the group: states, y, and dC's products.
        coefficients(t0, 0, Bt, Ct);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (i + 2 < K) fetch(t0, i + 2);
            if (i + 1 < K) coefficients(t0, i + 1, Bn, Cn);
            if (i > 0) column_read();
            const uint32_t in = i < m ? live : 0u;
            float sig, r, gz, y = 0.f;
            const float dt = masked(sel_dt(to_f32(dv[i % 3]) + bias, softplus, &sig), in);
            const float u = masked(to_f32(uv[i % 3]), in), x = dt * u;
            upstream(dyv[i % 3], GATE ? zv[i % 3] : dyv[i % 3], in, &r, &gz);
            tok[wave / NB][i][0][lane] = dt;
            tok[wave / NB][i][1][lane] = u;
            tok[wave / NB][i][2][lane] = sig;
            tok[wave / NB][i][3][lane] = r;
            f32x4 p;
#pragma unroll
            for (int n = 0; n < kSB; ++n) {
                hs[i][n] = fmaf(exp2_fast(dt * A2[n]), i ? hs[i ? i - 1 : 0][n] : h0[n], x * Bt[n]);
                if (GATE) y = fmaf(Ct[n], hs[i][n], y);
                p[n & 3] = r * hs[i][n];
                if ((n & 3) == 3) *reinterpret_cast<f32x4 *>(mine + (n - 3)) = p;
            }
            if (i > 0) comb[wave][i - 1][1][lane] = column_sum();
            if constexpr (NB == 1) finish_z(t0 + i, u, r, gz, y);
            else {
                cross[wave][i][0][lane] = y;
            }
            Bt = Bn;
            Ct = Cn;
            __builtin_amdgcn_sched_barrier(0);
        }
        // A row that ends inside the group: the states from its last token on are what the copied
        // tokens would multiply by 0.
        if (m < K) {
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int n = 0; n < kSB; ++n) hs[i][n] = masked(hs[i][n], i < m - 1 ? ~0u : 0u);
        }
        // And back: g, what follows from it, and dB's products.
        coefficients(t0, K - 1, Bt, Ct);
#pragma unroll
        for (int i = K - 1; i >= 0; --i) {
            if (i > 0) coefficients(t0, i - 1, Bn, Cn);
            if (i == 2) kept_state(hidden(t0), h0);         // again, now that later tokens' states are done with
            if (i == 1) {                                   // what the next group starts with
                const int tp = hidden(max(t0 - K, begin));
                kept_state(tp, hn);
                fetch(tp, 0);
                fetch(tp, 1);
            }
            column_read();
            const float dt = tok[wave / NB][i][0][back], u = tok[wave / NB][i][1][back], sig = tok[wave / NB][i][2][back];
            const float r = tok[wave / NB][i][3][back], x = dt * u;
            float qq = 0.f, dw = 0.f;
            f32x4 p;
#pragma unroll
            for (int n = 0; n < kSB; ++n) {
                const float gg = fmaf(r, Ct[n], carry[n]);
                qq = fmaf(gg, Bt[n], qq);
                p[n & 3] = gg * x;
                carry[n] = exp2_fast(dt * A2[n]) * gg;
                const float w = carry[n] * (i ? hs[i ? i - 1 : 0][n] : h0[n]);
                dw = fmaf(w, A2[n], dw);
                dA[n] = fmaf(w, dt, dA[n]);
                pinned(dA[n]);
                if ((n & 3) == 3) *reinterpret_cast<f32x4 *>(mine + (n - 3)) = p;
            }
            const float s = column_sum();
            if (i == K - 1) comb[wave][K - 1][1][lane] = s;
            else comb[wave][i + 1][0][lane] = s;
            if constexpr (NB == 1) finish_u(t0 + i, dt, u, sig, r, qq, dw);
            else {
                cross[wave][i][1][lane] = qq;
                cross[wave][i][2][lane] = dw;
            }
            Bt = Bn;
            Ct = Cn;
            __builtin_amdgcn_sched_barrier(0);
        }
        column_read();
        comb[wave][0][0][lane] = column_sum();
        __syncthreads();
        // dB, dC of the 8 tokens: the sums of the workgroup's tiles and lane quarters
#pragma unroll
        for (int e = threadIdx.x; e < K * 32 * NB; e += 256) {
            const int v = e % 16, which = e / 16 % 2, i = e / 32 % K, k = e / 32 / K;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < TPB; ++w) {
                const float *p = comb[w * NB + k][i][which] + v;
                s += (p[0] + p[16]) + (p[32] + p[48]);
            }
            if (i < m)
                a.part_bc[(((((int64_t)part * a.batch + b) * a.L + t0 + i) * a.G + g) * 2 + which) * N + k * kSB + v] = s;
        }
        if constexpr (NB > 1) {
            // the tile's NB waves share out its tokens, each adding the blocks' parts
            for (int i = nb; i < K; i += NB) {
                float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NB; ++w)
#pragma unroll
                    for (int k = 0; k < 3; ++k) s[k] += cross[wave - nb + w][i][k][lane];
                const int t = min(t0 + i, end - 1);
                float r, gz;
                T dy1 = lane_load(r_dy.at(t), d), z1 = dy1;
                if (GATE) z1 = lane_load(r_z.at(t), d);
                upstream(dy1, z1, i < m ? live : 0u, &r, &gz);
                finish_z(t0 + i, tok[wave / NB][i][1][lane], r, gz, s[0]);
                finish_u(t0 + i, tok[wave / NB][i][0][lane], tok[wave / NB][i][1][lane], tok[wave / NB][i][2][lane], r, s[1], s[2]);
            }
        }
        __syncthreads();
    }
    if (q.live) {
        for (int t = max(begin, end) + nb; t < stop; t += NB) {
            lane_store(out_row(a.du, t), d, from_f32<T>(0.f));
            lane_store(out_row(a.ddelta, t), d, from_f32<T>(0.f));
            if (GATE) lane_store(out_row(a.dz, t), d, from_f32<T>(0.f));
        }
        if (c == 0 && a.dinit) {
            float *o = a.dinit + (b * a.D + q.d) * (int64_t)N + n0;
#pragma unroll
            for (int n = 0; n < kSB; ++n) o[n] = carry[n];
        }
    }
    // sums over this chunk's tokens; dD and dbias are spread over the blocks of states
    if constexpr (NB > 1) {
        comb[wave][0][0][lane] = dD;
        comb[wave][0][1][lane] = dbias;
        __syncthreads();
        dD = dbias = 0.f;
#pragma unroll
        for (int w = 0; w < NB; ++w) {
            dD += comb[wave - nb + w][0][0][lane];
            dbias += comb[wave - nb + w][0][1][lane];
        }
    }
    if (real) {
        float *o = a.part_par + sel_slot(a, b, c, q.tt, N + 2);
#pragma unroll
        for (int n = 0; n < kSB; ++n) o[(n0 + n) * 64] = dA[n];
        if (nb == 0) {
            o[N * 64] = dD;
            o[(N + 1) * 64] = dbias;
        }
    }
}

// dB and dC: partial sums added in order, rounded once; tokens past a row's end are zero.
template <typename T>
__global__ __launch_bounds__(256) void sel_bwd_bc_kernel(SelArgs a, int parts) {
    const int64_t gn = (int64_t)a.G * a.N, per = a.batch * a.L * gn * 2;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= per) return;
    const int n = (int)(k % a.N), which = (int)(k / a.N % 2), g = (int)(k / a.N / 2 % a.G);
    const int64_t bt = k / a.N / 2 / a.G, b = bt / a.L;
    const int t = (int)(bt % a.L);
    float s = 0.f;
    if (t < row_length(a.lengths, b, a.L))
        for (int p = 0; p < parts; ++p) s += a.part_bc[p * per + k];
    reinterpret_cast<T *>(which ? a.dC : a.dB)[bt * gn + g * a.N + n] = from_f32<T>(s);
}

// dA, dD and dbias: partial sums of all (batch row, chunk).
__global__ __launch_bounds__(1024) void sel_bwd_par_kernel(SelArgs a) {
    __shared__ float red[16][64];
    const int n = blockIdx.x % (a.N + 2), tt = blockIdx.x / (a.N + 2);
    const SelTile q = sel_tile(a, tt);
    const float s = rows_sum<16>(a.part_par + ((int64_t)tt * (a.N + 2) + n) * 64 + threadIdx.x % 64, a.batch * a.nc,
                                 (int64_t)a.G * a.tiles * (a.N + 2) * 64, red);
    if (threadIdx.x >= 64 || !q.live) return;
    if (n < a.N) a.dA[(int64_t)q.d * a.N + n] = s;
    else if (n == a.N) { if (a.dD) a.dD[q.d] = s; }
    else if (a.dbias) a.dbias[q.d] = s;
}

template <typename T, int N>
static hipError_t sel_bwd_t(const SelArgs &a, hipStream_t s) {
    const int parts = sel_bwd_parts(a.D, a.G, N);
    const int64_t blocks = a.batch * a.nc * a.G * parts;
    const int64_t sums = (a.batch * a.L * a.G * a.N * 2 + 255) / 256;
    const int64_t pars = (int64_t)a.G * a.tiles * (N + 2);
    if (!grid_fits(blocks, 256) || !grid_fits(sums, 256) || !grid_fits(pars, 1024)) return hipErrorInvalidValue;
    hipError_t e;
    if (a.nc > 1) {
        if ((e = launch_sel_local_reverse(a, s)) != hipSuccess) return e;
        if ((e = launch_sel_pass(a, true, s)) != hipSuccess) return e;
    }
    if (a.z.p) sel_bwd_kernel<T, N, true><<<(uint32_t)blocks, 256, 0, s>>>(a);
    else sel_bwd_kernel<T, N, false><<<(uint32_t)blocks, 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sel_bwd_bc_kernel<T><<<(uint32_t)sums, 256, 0, s>>>(a, parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sel_bwd_par_kernel<<<(uint32_t)pars, 1024, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_sel_bwd(const SelArgs &a, hipStream_t s) {
    if (a.dtype == 1) {
        if (a.N == 16) return sel_bwd_t<bf16, 16>(a, s);
        if (a.N == 32) return sel_bwd_t<bf16, 32>(a, s);
        if (a.N == 64) return sel_bwd_t<bf16, 64>(a, s);
    } else {
        if (a.N == 16) return sel_bwd_t<float, 16>(a, s);
        if (a.N == 32) return sel_bwd_t<float, 32>(a, s);
        if (a.N == 64) return sel_bwd_t<float, 64>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace ssd
