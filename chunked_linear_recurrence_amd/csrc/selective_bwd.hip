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
// The forward leaves the state before every 8th token.  From the last group of 8 tokens to
// the first, a wave (64 channels, one lane each, 16 states) runs the group forward from that
// state, keeping its 8 states in registers, and then backward through them.  h_{t-1} is
// never recovered by division, which would lose it where decays are small.  The decays are
// computed a second time on the way back: keeping them too would take twice the registers
// and leave one wave per SIMD.
//
// The sums over channels (dB, dC: 32 values a token) go through LDS: every lane writes its
// 32 products, and each lane then adds half a column.  The 4 waves of a workgroup are 64/N
// tiles times N/16 blocks of states; their sums meet in LDS, and one partial sum per
// workgroup goes to memory, added up in order by a last kernel, so that results do not
// depend on scheduling.
#include "ssd_sel.h"

namespace ssd {

constexpr int kSB = 16;               // states per wave
constexpr int kRow = 36;              // floats per lane in the reduction buffer: 32 and padding, 16-byte rows
constexpr int kHalf = 32 * kRow + 32; // second half of the lanes: 32 banks away from the first

template <typename T, int N>
__global__ __launch_bounds__(256, 2) void sel_bwd_kernel(SelArgs a) {
    constexpr int NB = N / kSB, TPB = 4 / NB, K = kKeep;
    __shared__ float red[4][2 * kHalf];
    __shared__ float comb[4][K][64];
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
    sel_rates<kSB>(a, q.d, n0, A2);
    const float *S = a.S + sel_slot(a, b, c, q.tt, N) + n0 * 64;
    const float *f0 = a.dfinal ? a.dfinal + (b * a.D + q.d) * (int64_t)N + n0 : nullptr;
#pragma unroll
    for (int n = 0; n < kSB; ++n) {
        carry[n] = a.nc > 1 ? S[n * 64] : (f0 ? f0[n] : 0.f);
        dA[n] = 0.f;
    }
    T *du = reinterpret_cast<T *>(a.du) + b * a.L * (int64_t)a.D + q.d;
    T *dd = reinterpret_cast<T *>(a.ddelta) + b * a.L * (int64_t)a.D + q.d;
    T *dz = reinterpret_cast<T *>(a.dz) + b * a.L * (int64_t)a.D + q.d;

    for (int t0 = begin + (max(end - begin, 1) - 1) / K * K; t0 >= begin && t0 < end; t0 -= K) {
        const int m = min(K, end - t0);
        float dt[K], u[K], sig[K], r[K], gz[K], yp[K], qs[K], ds[K], rs[K];
        float h0[kSB], hs[K][kSB];
        const float *kp = a.keep + sel_keep_slot(a, b, t0 / K, q.tt, n0);
#pragma unroll
        for (int n = 0; n < kSB; ++n) h0[n] = kp[n * 64];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int t = min(t0 + i, end - 1);
            const bool in = q.live && i < m;                // others add nothing to any sum
            const float dy = to_f32(row_of<T>(a.dy, b, t)[q.d]);
            const float raw = to_f32(row_of<T>(a.delta, b, t)[q.d]) + bias;
            u[i] = in ? to_f32(row_of<T>(a.u, b, t)[q.d]) : 0.f;
            dt[i] = sel_dt(raw, softplus, &sig[i]);
            dt[i] = in ? dt[i] : 0.f;
            r[i] = in ? dy : 0.f;
            gz[i] = 0.f;
            if (a.z.p) {
                const float z = to_f32(row_of<T>(a.z, b, t)[q.d]);
                gz[i] = r[i] * dsilu_f32(z);
                r[i] = in ? r[i] * silu_f32(z) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int t = min(t0 + i, end - 1);
            Uniform<T, kSB> Bt, Ct;
            Bt.load(row_of<T>(a.B, b, t) + g * N + n0);
            Ct.load(row_of<T>(a.C, b, t) + g * N + n0);
            const float x = dt[i] * u[i];
            float y = 0.f;
#pragma unroll
            for (int n = 0; n < kSB; ++n) {
                hs[i][n] = fmaf(exp2_fast(dt[i] * A2[n]), i ? hs[i ? i - 1 : 0][n] : h0[n], x * Bt[n]);
                y = fmaf(Ct[n], hs[i][n], y);
            }
            yp[i] = y;
        }
        float *mine = red[wave] + (lane / 32) * kHalf + (lane % 32) * kRow;
        const float *column = red[wave] + (lane / 32) * kHalf + lane % 32;
#pragma unroll
        for (int i = K - 1; i >= 0; --i) {
            const int t = min(t0 + i, end - 1);
            Uniform<T, kSB> Bt, Ct;
            Bt.load(row_of<T>(a.B, b, t) + g * N + n0);
            Ct.load(row_of<T>(a.C, b, t) + g * N + n0);
            const float x = dt[i] * u[i];
            float qq = 0.f, dw = 0.f;
            f32x4 pb, pc;
#pragma unroll
            for (int n = 0; n < kSB; ++n) {
                const float gg = fmaf(r[i], Ct[n], carry[n]);
                qq = fmaf(gg, Bt[n], qq);
                pb[n & 3] = gg * x;
                pc[n & 3] = r[i] * hs[i][n];
                carry[n] = exp2_fast(dt[i] * A2[n]) * gg;
                const float w = carry[n] * (i ? hs[i ? i - 1 : 0][n] : h0[n]);
                dw = fmaf(w, A2[n], dw);
                dA[n] = fmaf(w, dt[i], dA[n]);
                if ((n & 3) == 3) {
                    *reinterpret_cast<f32x4 *>(mine + (n - 3)) = pb;
                    *reinterpret_cast<f32x4 *>(mine + 16 + (n - 3)) = pc;
                }
            }
            qs[i] = qq;
            ds[i] = dw;
            __builtin_amdgcn_wave_barrier();
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                s0 += column[k * kRow];
                s1 += column[(k + 1) * kRow];
            }
            rs[i] = s0 + s1;
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int i = 0; i < K; ++i) comb[wave][i][lane] = rs[i];
        if constexpr (NB > 1) {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                cross[wave][i][0][lane] = yp[i];
                cross[wave][i][1][lane] = qs[i];
                cross[wave][i][2][lane] = ds[i];
            }
        }
        __syncthreads();
        // dB, dC of the 8 tokens: the sums of the workgroup's tiles and lane halves
#pragma unroll
        for (int e = threadIdx.x; e < K * 32 * NB; e += 256) {
            const int v = e % 32, i = e / 32 % K, k = e / 32 / K;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < TPB; ++w) s += comb[w * NB + k][i][v] + comb[w * NB + k][i][32 + v];
            if (i < m)
                a.part_bc[(((((int64_t)part * a.batch + b) * a.L + t0 + i) * a.G + g) * 2 + v / 16) * N + k * kSB + v % 16] = s;
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if (i % NB == nb) {
                if constexpr (NB > 1) {
                    yp[i] = qs[i] = ds[i] = 0.f;
                    const int w0 = wave - nb;
#pragma unroll
                    for (int w = 0; w < NB; ++w) {
                        yp[i] += cross[w0 + w][i][0][lane];
                        qs[i] += cross[w0 + w][i][1][lane];
                        ds[i] += cross[w0 + w][i][2][lane];
                    }
                }
                const float dl = fmaf(ds[i], kLn2F, u[i] * qs[i]) * sig[i];
                dD = fmaf(r[i], u[i], dD);
                if (q.live && i < m) {
                    const int64_t at = (t0 + i) * (int64_t)a.D;
                    dbias += dl;
                    du[at] = from_f32<T>(fmaf(dt[i], qs[i], skip * r[i]));
                    dd[at] = from_f32<T>(dl);
                    if (a.z.p) dz[at] = from_f32<T>(gz[i] * fmaf(skip, u[i], yp[i]));
                }
            }
        }
        __syncthreads();
    }
    if (q.live) {
        for (int t = max(begin, end) + nb; t < stop; t += NB) {
            const int64_t at = t * (int64_t)a.D;
            du[at] = dd[at] = from_f32<T>(0.f);
            if (a.z.p) dz[at] = from_f32<T>(0.f);
        }
        if (c == 0 && a.dinit) {
            float *o = a.dinit + (b * a.D + q.d) * (int64_t)N + n0;
#pragma unroll
            for (int n = 0; n < kSB; ++n) o[n] = carry[n];
        }
    }
    // sums over this chunk's tokens; dD and dbias are spread over the blocks of states
    if constexpr (NB > 1) {
        cross[wave][0][0][lane] = dD;
        cross[wave][0][1][lane] = dbias;
        __syncthreads();
        dD = dbias = 0.f;
#pragma unroll
        for (int w = 0; w < NB; ++w) {
            dD += cross[wave - nb + w][0][0][lane];
            dbias += cross[wave - nb + w][0][1][lane];
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

// dA, dD and dbias: partial sums of all (batch row, chunk), 4 quarters of them in order.
__global__ __launch_bounds__(256) void sel_bwd_par_kernel(SelArgs a) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x % 64, k = threadIdx.x / 64;
    const int n = blockIdx.x % (a.N + 2), tt = blockIdx.x / (a.N + 2);
    const SelTile q = sel_tile(a, tt);
    const int64_t rows = a.batch * a.nc, rs = (int64_t)a.G * a.tiles * (a.N + 2) * 64;
    const float *p = a.part_par + ((int64_t)tt * (a.N + 2) + n) * 64 + lane;
    float s = 0.f;
    for (int64_t r = rows * k / 4; r < rows * (k + 1) / 4; ++r) s += p[r * rs];
    red[k][lane] = s;
    __syncthreads();
    if (k == 0 && q.live) {
        s = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
        if (n < a.N) a.dA[(int64_t)q.d * a.N + n] = s;
        else if (n == a.N) { if (a.dD) a.dD[q.d] = s; }
        else if (a.dbias) a.dbias[q.d] = s;
    }
}

template <typename T, int N>
static hipError_t sel_bwd_t(const SelArgs &a, hipStream_t s) {
    const int parts = sel_bwd_parts(a.D, a.G, N);
    hipError_t e;
    if (a.nc > 1) {
        if ((e = launch_sel_local_reverse(a, s)) != hipSuccess) return e;
        if ((e = launch_sel_pass(a, true, s)) != hipSuccess) return e;
    }
    const int64_t blocks = a.batch * a.nc * a.G * parts;
    const int64_t sums = (a.batch * a.L * a.G * a.N * 2 + 255) / 256;
    const int64_t pars = (int64_t)a.G * a.tiles * (N + 2);
    if (blocks > INT32_MAX || sums > INT32_MAX || pars > INT32_MAX) return hipErrorInvalidValue;
    sel_bwd_kernel<T, N><<<(uint32_t)blocks, 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sel_bwd_bc_kernel<T><<<(uint32_t)sums, 256, 0, s>>>(a, parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sel_bwd_par_kernel<<<(uint32_t)pars, 256, 0, s>>>(a);
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
