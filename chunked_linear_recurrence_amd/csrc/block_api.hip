// C-ABI entry points of the operators around a scan: short causal convolution, selective
// scan and layer norm.  Argument checks, workspace carving and launches on the caller's
// stream; nothing here allocates device memory or waits on the device.
#include "libssdscan.h"

#include <math.h>
#include <string.h>

#include "ssd_block.h"
#include "ssd_entry.h"

using namespace ssd_check;

namespace {

// The dims with the strides over dimensions of one element, which nothing uses, as 0: they are
// neither checked nor looked at where a kernel is chosen.
ssd_conv_dims_t used(ssd_conv_dims_t d) {
    if (d.batch == 1) d.x_batch_stride = d.dy_batch_stride = 0;
    if (d.seqlen == 1) d.x_token_stride = d.dy_token_stride = 0;
    return d;
}
ssd_selective_dims_t used(ssd_selective_dims_t d) {
    if (d.batch == 1)
        d.u_batch_stride = d.delta_batch_stride = d.z_batch_stride = d.B_batch_stride = d.C_batch_stride =
            d.dy_batch_stride = 0;
    if (d.seqlen == 1)
        d.u_token_stride = d.delta_token_stride = d.z_token_stride = d.B_token_stride = d.C_token_stride =
            d.dy_token_stride = 0;
    return d;
}
ssd_norm_dims_t used(ssd_norm_dims_t d) {
    if (d.rows == 1) d.x_row_stride = d.dy_row_stride = 0;
    return d;
}

// ------------------------------------------------------------------------- convolution
ssd_status_t check_conv(const ssd_conv_dims_t *d, bool step) {
    if (!d) return fail(SSD_ERR_NULL_ARG, "dims is NULL");
    TRY(check_dtype(d->dtype));
    if (d->batch <= 0 || d->seqlen <= 0 || d->channels <= 0)
        return fail(SSD_ERR_BAD_SHAPE, "every dimension must be >= 1 (batch %lld seqlen %lld channels %lld)",
                    (long long)d->batch, (long long)d->seqlen, (long long)d->channels);
    if (step && d->seqlen != 1)
        return fail(SSD_ERR_BAD_SHAPE, "a step takes one token: seqlen must be 1 (got %lld)", (long long)d->seqlen);
    if (d->width < 1) return fail(SSD_ERR_BAD_SHAPE, "width must be >= 1 (got %d)", d->width);
    if (!ssd::conv_supported(d->width))
        return fail(SSD_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %d)", d->width);
    if (d->seqlen > INT32_MAX / 2 || d->channels > INT32_MAX / 16)
        return fail(SSD_ERR_UNSUPPORTED, "seqlen or channels exceed the kernels' index range");
    int64_t n;
    if (!product({d->batch, d->seqlen + d->width, d->channels}, &n)) return fail(SSD_ERR_BAD_SHAPE, "sizes overflow");
    return SSD_OK;
}

ssd::ConvArgs conv_args(const ssd_conv_dims_t &d, const void *x, const float *w, const float *bias, const void *init,
                        const int32_t *lengths, uint32_t flags) {
    ssd::ConvArgs a;
    memset(&a, 0, sizeof(a));
    a.batch = d.batch;
    a.L = (int)d.seqlen;
    a.C = (int)d.channels;
    a.W = d.width;
    a.dtype = d.dtype;
    a.flags = flags;
    a.x = {x, d.x_batch_stride, d.x_token_stride};
    a.w = w;
    a.bias = bias;
    a.init = init;
    a.lengths = lengths;
    return a;
}

size_t conv_ws(const ssd_conv_dims_t &d) {
    int64_t n;
    if (!product({ssd::conv_bwd_rows(d.batch, d.seqlen, d.channels, d.dtype), d.width + 1, d.channels, 4}, &n)) return 0;
    return align_up((size_t)n);
}

// ----------------------------------------------------------------------- selective scan
ssd_status_t check_sel(const ssd_selective_dims_t *d, bool step) {
    if (!d) return fail(SSD_ERR_NULL_ARG, "dims is NULL");
    TRY(check_dtype(d->dtype));
    if (d->reserved != 0) return fail(SSD_ERR_BAD_SHAPE, "dims.reserved must be 0");
    if (d->batch <= 0 || d->seqlen <= 0 || d->channels <= 0 || d->dstate <= 0 || d->ngroups <= 0)
        return fail(SSD_ERR_BAD_SHAPE, "every dimension must be >= 1 (batch %lld seqlen %lld channels %lld dstate "
                    "%lld ngroups %lld)", (long long)d->batch, (long long)d->seqlen, (long long)d->channels,
                    (long long)d->dstate, (long long)d->ngroups);
    if (d->channels % d->ngroups != 0)
        return fail(SSD_ERR_BAD_SHAPE, "channels %lld is not a multiple of ngroups %lld", (long long)d->channels,
                    (long long)d->ngroups);
    if (step && d->seqlen != 1)
        return fail(SSD_ERR_BAD_SHAPE, "a step takes one token: seqlen must be 1 (got %lld)", (long long)d->seqlen);
    if (!ssd::sel_supported(d->dstate))
        return fail(SSD_ERR_UNSUPPORTED, "dstate must be 16, 32 or 64 (got %lld)", (long long)d->dstate);
    if (d->seqlen > INT32_MAX / 2 || d->channels > INT32_MAX / 256)
        return fail(SSD_ERR_UNSUPPORTED, "seqlen or channels exceed the kernels' index range");
    int64_t n;
    // every tensor and workspace is below 4 float32 per (token, padded channel, state)
    if (!product({d->batch, d->seqlen + 64, d->channels + 64 * d->ngroups, d->dstate + 2, 8}, &n))
        return fail(SSD_ERR_BAD_SHAPE, "sizes overflow");
    return SSD_OK;
}

// How a sequence is cut into chunks: waves that the chunks come to together (8 for each of 1024
// SIMDs in the forward, 4 in the backward), and from how many waves of a single pass on, and up
// to how many tokens, one pass is taken.  Fewer are resident at a time: (3) takes 72 registers
// with 16 states in bfloat16 (7 waves a SIMD; 5 in float32), 108 to 123 with 32 (4) and 188 to
// 219 with 64 (2); the backward's large kernel holds 2.  Measured with 16 states in bfloat16
// alone, and taken for the other sizes as it is.  Waves: 32768 tokens of 2048 channels take 572 us with 2048
// waves, 443 with 4096, 401 with 8192, 406 with 12288; forward and backward of 2 x 4096 tokens
// 464, 433, 434, 440 by the forward's, and 443, 434, - and 444 by the backward's.  One pass, 256
// and 1024 tokens of 2048 channels: 143 and 562 us with 1280 waves against 137 and 467 in chunks,
// 142 and 562 with 1536 against 176 and 556, 144 and 564 with 1792 against 190 and 621; with the
// backward 604 and 2355 with 1536 against 653 and 2155, 612 and 2405 with 1792 against 721 and
// 2475.  32 tokens of 1536 channels: 16.6 us in one pass against 20.5 (48 tokens: 23.4, 20.2).
constexpr ssd::SelCut kSelFwd = {8192, 1536, 32}, kSelBwd = {4096, 1792, 16};

ssd::SelArgs sel_args(const ssd_selective_dims_t &d, bool backward) {
    ssd::SelArgs a;
    memset(&a, 0, sizeof(a));
    a.batch = d.batch;
    a.L = (int)d.seqlen;
    a.D = (int)d.channels;
    a.N = (int)d.dstate;
    a.G = (int)d.ngroups;
    a.dtype = d.dtype;
    a.tiles = ssd::sel_tiles(d.channels, d.ngroups);
    const int64_t waves = backward ? d.batch * d.ngroups * ssd::sel_bwd_parts(d.channels, d.ngroups, d.dstate) * 4
                                   : d.batch * d.ngroups * a.tiles;
    ssd::sel_chunks(waves, backward ? kSelBwd : kSelFwd, d.seqlen, &a.nc, &a.T);
    return a;
}

struct SelLayout {
    size_t S, sumdt, bc, par, total;
};

SelLayout sel_layout(const ssd::SelArgs &a, bool backward) {
    SelLayout lo;
    const size_t slots = (size_t)a.batch * a.nc * a.G * a.tiles * 64 * 4;
    size_t off = 0;
    lo.S = off;
    if (a.nc > 1) off += align_up(slots * a.N);
    lo.sumdt = off;
    if (a.nc > 1) off += align_up(slots);
    lo.bc = lo.par = off;
    if (backward) {
        off += align_up((size_t)ssd::sel_bwd_parts(a.D, a.G, a.N) * a.batch * a.L * a.G * 2 * a.N * 4);
        lo.par = off;
        off += align_up(slots * (a.N + 2));
    }
    lo.total = off;
    return lo;
}

size_t sel_kept(const ssd_selective_dims_t &d) {
    const int64_t nsub = (d.seqlen + ssd::kKeep - 1) / ssd::kKeep;
    return (size_t)(d.batch * nsub * d.ngroups * ssd::sel_tiles(d.channels, d.ngroups) * d.dstate) * 64 * 4;
}

// Bytes spanned by u, delta, z, B, C and dy, in this order; 0 for one that is not there, whose
// strides are not looked at.
ssd_status_t sel_spans(const ssd_selective_dims_t &d, const void *z, const void *dy, bool step, size_t out[6]) {
    const int64_t e = act_bytes(d.dtype), gn = d.ngroups * d.dstate;
    const int64_t bs[] = {d.u_batch_stride, d.delta_batch_stride, d.z_batch_stride, d.B_batch_stride, d.C_batch_stride,
                          d.dy_batch_stride};
    const int64_t ts[] = {d.u_token_stride, d.delta_token_stride, d.z_token_stride, d.B_token_stride, d.C_token_stride,
                          d.dy_token_stride};
    for (int i = 0; i < 6; ++i) {
        out[i] = 0;
        if ((i == 2 && !z) || (i == 5 && !dy)) continue;
        const int64_t t = ts[i];
        const bool coef = i == 3 || i == 4;
        if (!span(d.batch, bs[i], d.seqlen, t, coef ? gn : d.channels, e, &out[i]))
            return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
        if (t > INT32_MAX / e) return fail(SSD_ERR_UNSUPPORTED, "a token stride spans more than 2^31 bytes");
        if (coef && !step && e == 2 && ((bs[i] | t) & 1))
            return fail(SSD_ERR_MISALIGNED, "bfloat16 B and C need even strides (4-byte rows)");
    }
    return SSD_OK;
}

// ------------------------------------------------------------------------------- norm
ssd_status_t check_norm(const ssd_norm_dims_t *d) {
    if (!d) return fail(SSD_ERR_NULL_ARG, "dims is NULL");
    TRY(check_dtype(d->dtype));
    if (d->reserved != 0) return fail(SSD_ERR_BAD_SHAPE, "dims.reserved must be 0");
    if (d->rows <= 0 || d->channels <= 0)
        return fail(SSD_ERR_BAD_SHAPE, "every dimension must be >= 1 (rows %lld channels %lld)", (long long)d->rows,
                    (long long)d->channels);
    if (d->channels > INT32_MAX / 16) return fail(SSD_ERR_UNSUPPORTED, "channels exceed the kernels' index range");
    int64_t n;
    if (!product({d->rows, d->channels}, &n)) return fail(SSD_ERR_BAD_SHAPE, "sizes overflow");
    return SSD_OK;
}

size_t norm_ws(const ssd_norm_dims_t &d) {
    return align_up((size_t)ssd::norm_bwd_blocks(d.rows) * 2 * (size_t)d.channels * 4);
}

}  // namespace

extern "C" {

ssd_status_t ssd_conv_fwd(const ssd_conv_dims_t *dims, const void *x, const float *weight, const float *bias,
                          const void *init_state, const int32_t *lengths, void *y, void *final_state, uint32_t flags,
                          void *stream) {
    TRY(check_conv(dims, false));
    const ssd_conv_dims_t d = used(*dims);
    if (!x || !weight || !y) return fail(SSD_ERR_NULL_ARG, "x, weight and y must be non-NULL");
    if (flags & ~SSD_FLAG_SILU) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    const size_t e = (size_t)act_bytes(d.dtype), C = (size_t)d.channels;
    size_t nx;
    if (!span(d.batch, d.x_batch_stride, d.seqlen, d.x_token_stride, d.channels, e, &nx))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const size_t ny = (size_t)(d.batch * d.seqlen) * C * e, ns = (size_t)(d.batch * (d.width - 1)) * C * e;
    const bool in_place = init_state && init_state == final_state;
    const Tensor in[] = {{"x", x, nx, e}, {"weight", weight, C * d.width * 4, 4}, {"bias", bias, C * 4, 4},
                         {"lengths", lengths, (size_t)d.batch * 4, 4},
                         {"init_state", in_place ? nullptr : init_state, ns, e}};
    const Tensor out[] = {{"y", y, ny, e}, {"final_state", final_state, ns, e}};
    TRY(check_tensors(in, 5, out, 2));
    ssd::ConvArgs a = conv_args(d, x, weight, bias, init_state, lengths, flags);
    a.y = y;
    a.final_state = final_state;
    return launched("ssd_conv_fwd", ssd::launch_conv_fwd(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_conv_step(const ssd_conv_dims_t *dims, const void *x, const float *weight, const float *bias,
                           const void *state_in, void *state_out, void *y, uint32_t flags, void *stream) {
    TRY(check_conv(dims, true));
    const ssd_conv_dims_t d = used(*dims);
    if (!x || !weight || !state_in || !state_out || !y)
        return fail(SSD_ERR_NULL_ARG, "x, weight, state_in, state_out and y must be non-NULL");
    if (flags & ~SSD_FLAG_SILU) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    const size_t e = (size_t)act_bytes(d.dtype), C = (size_t)d.channels;
    size_t nx;
    if (!span(d.batch, d.x_batch_stride, 1, 0, d.channels, e, &nx))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const size_t ns = (size_t)(d.batch * (d.width - 1)) * C * e;
    const Tensor in[] = {{"x", x, nx, e}, {"weight", weight, C * d.width * 4, 4}, {"bias", bias, C * 4, 4},
                         {"state_in", state_in == state_out ? nullptr : state_in, ns, e}};
    const Tensor out[] = {{"y", y, (size_t)d.batch * C * e, e}, {"state_out", state_out, ns, e}};
    TRY(check_tensors(in, 4, out, 2));
    ssd::ConvArgs a = conv_args(d, x, weight, bias, state_in, nullptr, flags);
    a.y = y;
    a.final_state = state_out;
    return launched("ssd_conv_step", ssd::launch_conv_step(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_conv_bwd_workspace_bytes(const ssd_conv_dims_t *dims) {
    return check_conv(dims, false) == SSD_OK ? conv_ws(*dims) : 0;
}

ssd_status_t ssd_conv_bwd(const ssd_conv_dims_t *dims, const void *dy, const void *x, const float *weight,
                          const float *bias, const void *init_state, const void *dfinal, const int32_t *lengths,
                          void *dx, float *dweight, float *dbias, void *dinit, uint32_t flags, void *workspace,
                          size_t workspace_bytes, void *stream) {
    TRY(check_conv(dims, false));
    const ssd_conv_dims_t d = used(*dims);
    if (!dy || !x || !weight || !dx || !dweight)
        return fail(SSD_ERR_NULL_ARG, "dy, x, weight, dx and dweight must be non-NULL");
    if (flags & ~SSD_FLAG_SILU) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    const size_t need = conv_ws(d);
    if (!need) return fail(SSD_ERR_BAD_SHAPE, "sizes overflow");
    if (!workspace || workspace_bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace %p of %zu bytes; %zu bytes are needed", workspace, workspace_bytes, need);
    const size_t e = (size_t)act_bytes(d.dtype), C = (size_t)d.channels;
    size_t nx, ng;
    if (!span(d.batch, d.x_batch_stride, d.seqlen, d.x_token_stride, d.channels, e, &nx) ||
        !span(d.batch, d.dy_batch_stride, d.seqlen, d.dy_token_stride, d.channels, e, &ng))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const size_t ny = (size_t)(d.batch * d.seqlen) * C * e, ns = (size_t)(d.batch * (d.width - 1)) * C * e;
    const Tensor in[] = {{"dy", dy, ng, e}, {"x", x, nx, e}, {"weight", weight, C * d.width * 4, 4},
                         {"bias", bias, C * 4, 4}, {"lengths", lengths, (size_t)d.batch * 4, 4},
                         {"init_state", init_state, ns, e}, {"dfinal", dfinal, ns, e}};
    const Tensor out[] = {{"dx", dx, ny, e}, {"dweight", dweight, C * d.width * 4, 4}, {"dbias", dbias, C * 4, 4},
                          {"dinit", dinit, ns, e}, {"workspace", workspace, need, 16}};
    TRY(check_tensors(in, 7, out, 5));
    ssd::ConvArgs a = conv_args(d, x, weight, bias, init_state, lengths, flags);
    a.dy = {dy, d.dy_batch_stride, d.dy_token_stride};
    a.dfinal = dfinal;
    a.dx = dx;
    a.dinit = dinit;
    a.dw = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    return launched("ssd_conv_bwd", ssd::launch_conv_bwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_selective_kept_bytes(const ssd_selective_dims_t *dims) {
    return check_sel(dims, false) == SSD_OK ? sel_kept(*dims) : 0;
}

size_t ssd_selective_fwd_workspace_bytes(const ssd_selective_dims_t *dims) {
    if (check_sel(dims, false) != SSD_OK) return 0;
    return sel_layout(sel_args(*dims, false), false).total;
}

size_t ssd_selective_bwd_workspace_bytes(const ssd_selective_dims_t *dims) {
    if (check_sel(dims, false) != SSD_OK) return 0;
    return sel_layout(sel_args(*dims, true), true).total;
}

ssd_status_t ssd_selective_fwd(const ssd_selective_dims_t *dims, const void *u, const void *delta, const float *A,
                               const void *B, const void *C, const float *D, const void *z, const float *delta_bias,
                               const float *init_state, const int32_t *lengths, void *y, float *final_state, void *kept,
                               uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
    TRY(check_sel(dims, false));
    const ssd_selective_dims_t d = used(*dims);
    if (!u || !delta || !A || !B || !C || !y)
        return fail(SSD_ERR_NULL_ARG, "u, delta, A, B, C and y must be non-NULL");
    if (flags & ~SSD_FLAG_SOFTPLUS) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    size_t sp[6];
    TRY(sel_spans(d, z, nullptr, false, sp));
    ssd::SelArgs a = sel_args(d, false);
    const SelLayout lo = sel_layout(a, false);
    if (lo.total && (!workspace || workspace_bytes < lo.total))
        return fail(SSD_ERR_WORKSPACE, "workspace %p of %zu bytes; %zu bytes are needed", workspace, workspace_bytes,
                    lo.total);
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels;
    const size_t ns = (size_t)(d.batch * d.channels * d.dstate) * 4;
    const bool in_place = init_state && init_state == final_state;
    const Tensor in[] = {{"u", u, sp[0], e}, {"delta", delta, sp[1], e}, {"z", z, sp[2], e}, {"B", B, sp[3], 4},
                         {"C", C, sp[4], 4}, {"A", A, ch * d.dstate * 4, 4}, {"D", D, ch * 4, 4},
                         {"delta_bias", delta_bias, ch * 4, 4}, {"lengths", lengths, (size_t)d.batch * 4, 4},
                         {"init_state", in_place ? nullptr : init_state, ns, 4}};
    const Tensor out[] = {{"y", y, (size_t)(d.batch * d.seqlen) * ch * e, e}, {"final_state", final_state, ns, 4},
                          {"kept", kept, sel_kept(d), 16}, {"workspace", lo.total ? workspace : nullptr, lo.total, 16}};
    TRY(check_tensors(in, 10, out, 4));
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.flags = flags;
    a.u = {u, d.u_batch_stride, d.u_token_stride};
    a.delta = {delta, d.delta_batch_stride, d.delta_token_stride};
    a.z = {z, d.z_batch_stride, d.z_token_stride};
    a.B = {B, d.B_batch_stride, d.B_token_stride};
    a.C = {C, d.C_batch_stride, d.C_token_stride};
    a.A = A;
    a.Dskip = D;
    a.bias = delta_bias;
    a.init = init_state;
    a.lengths = lengths;
    a.y = y;
    a.final_state = final_state;
    a.keep = static_cast<float *>(kept);
    if (lo.total) {
        a.S = reinterpret_cast<float *>(ws + lo.S);
        a.sumdt = reinterpret_cast<float *>(ws + lo.sumdt);
    }
    return launched("ssd_selective_fwd", ssd::launch_sel_fwd(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_selective_step(const ssd_selective_dims_t *dims, const void *u, const void *delta, const float *A,
                                const void *B, const void *C, const float *D, const void *z, const float *delta_bias,
                                const float *state_in, float *state_out, void *y, uint32_t flags, void *stream) {
    TRY(check_sel(dims, true));
    const ssd_selective_dims_t d = used(*dims);
    if (!u || !delta || !A || !B || !C || !state_in || !state_out || !y)
        return fail(SSD_ERR_NULL_ARG, "u, delta, A, B, C, state_in, state_out and y must be non-NULL");
    if (flags & ~SSD_FLAG_SOFTPLUS) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    size_t sp[6];
    TRY(sel_spans(d, z, nullptr, true, sp));
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels;
    const size_t ns = (size_t)(d.batch * d.channels * d.dstate) * 4;
    if (!aligned16(state_in)) return fail(SSD_ERR_MISALIGNED, "state_in is not 16-byte aligned");
    const Tensor in[] = {{"u", u, sp[0], e}, {"delta", delta, sp[1], e}, {"z", z, sp[2], e}, {"B", B, sp[3], e},
                         {"C", C, sp[4], e}, {"A", A, ch * d.dstate * 4, 4}, {"D", D, ch * 4, 4},
                         {"delta_bias", delta_bias, ch * 4, 4},
                         {"state_in", state_in == state_out ? nullptr : state_in, ns, 16}};
    const Tensor out[] = {{"y", y, (size_t)d.batch * ch * e, e}, {"state_out", state_out, ns, 16}};
    TRY(check_tensors(in, 9, out, 2));
    ssd::SelStepArgs a;
    memset(&a, 0, sizeof(a));
    a.batch = d.batch;
    a.D = (int)d.channels;
    a.N = (int)d.dstate;
    a.G = (int)d.ngroups;
    a.dtype = d.dtype;
    a.flags = flags;
    a.u = u;
    a.u_bs = d.u_batch_stride;
    a.delta = delta;
    a.delta_bs = d.delta_batch_stride;
    a.z = z;
    a.z_bs = d.z_batch_stride;
    a.B = B;
    a.B_bs = d.B_batch_stride;
    a.C = C;
    a.C_bs = d.C_batch_stride;
    a.A = A;
    a.Dskip = D;
    a.bias = delta_bias;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    return launched("ssd_selective_step", ssd::launch_sel_step(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_selective_bwd(const ssd_selective_dims_t *dims, const void *dy, const void *u, const void *delta,
                               const float *A, const void *B, const void *C, const float *D, const void *z,
                               const float *delta_bias, const void *kept, const float *dfinal, const int32_t *lengths,
                               void *du, void *ddelta, float *dA, void *dB, void *dC, float *dD, void *dz,
                               float *ddelta_bias, float *dinit, uint32_t flags, void *workspace,
                               size_t workspace_bytes, void *stream) {
    TRY(check_sel(dims, false));
    const ssd_selective_dims_t d = used(*dims);
    if (!dy || !u || !delta || !A || !B || !C || !kept || !du || !ddelta || !dA || !dB || !dC)
        return fail(SSD_ERR_NULL_ARG, "dy, u, delta, A, B, C, kept, du, ddelta, dA, dB and dC must be non-NULL");
    if ((z != nullptr) != (dz != nullptr)) return fail(SSD_ERR_NULL_ARG, "dz must be given exactly if z is");
    if (flags & ~SSD_FLAG_SOFTPLUS) return fail(SSD_ERR_BAD_SHAPE, "unknown flag bits 0x%x", flags);
    size_t sp[6];
    TRY(sel_spans(d, z, dy, false, sp));
    ssd::SelArgs a = sel_args(d, true);
    const SelLayout lo = sel_layout(a, true);
    if (!workspace || workspace_bytes < lo.total)
        return fail(SSD_ERR_WORKSPACE, "workspace %p of %zu bytes; %zu bytes are needed", workspace, workspace_bytes,
                    lo.total);
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels;
    const size_t ns = (size_t)(d.batch * d.channels * d.dstate) * 4, ny = (size_t)(d.batch * d.seqlen) * ch * e;
    const size_t nbc = (size_t)(d.batch * d.seqlen * d.ngroups * d.dstate) * e;
    const Tensor in[] = {{"dy", dy, sp[5], e}, {"u", u, sp[0], e}, {"delta", delta, sp[1], e}, {"z", z, sp[2], e},
                         {"B", B, sp[3], 4}, {"C", C, sp[4], 4}, {"A", A, ch * d.dstate * 4, 4}, {"D", D, ch * 4, 4},
                         {"delta_bias", delta_bias, ch * 4, 4}, {"kept", kept, sel_kept(d), 16},
                         {"dfinal", dfinal, ns, 4}, {"lengths", lengths, (size_t)d.batch * 4, 4}};
    const Tensor out[] = {{"du", du, ny, e}, {"ddelta", ddelta, ny, e}, {"dz", dz, ny, e},
                          {"dA", dA, ch * d.dstate * 4, 4}, {"dB", dB, nbc, e}, {"dC", dC, nbc, e}, {"dD", dD, ch * 4, 4},
                          {"ddelta_bias", ddelta_bias, ch * 4, 4}, {"dinit", dinit, ns, 4},
                          {"workspace", workspace, lo.total, 16}};
    TRY(check_tensors(in, 12, out, 10));
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.flags = flags;
    a.dy = {dy, d.dy_batch_stride, d.dy_token_stride};
    a.u = {u, d.u_batch_stride, d.u_token_stride};
    a.delta = {delta, d.delta_batch_stride, d.delta_token_stride};
    a.z = {z, d.z_batch_stride, d.z_token_stride};
    a.B = {B, d.B_batch_stride, d.B_token_stride};
    a.C = {C, d.C_batch_stride, d.C_token_stride};
    a.A = A;
    a.Dskip = D;
    a.bias = delta_bias;
    a.lengths = lengths;
    a.keep = static_cast<float *>(const_cast<void *>(kept));
    a.dfinal = dfinal;
    a.du = du;
    a.ddelta = ddelta;
    a.dz = dz;
    a.dB = dB;
    a.dC = dC;
    a.dA = dA;
    a.dD = dD;
    a.dbias = ddelta_bias;
    a.dinit = dinit;
    a.S = reinterpret_cast<float *>(ws + lo.S);
    a.sumdt = reinterpret_cast<float *>(ws + lo.sumdt);
    a.part_bc = reinterpret_cast<float *>(ws + lo.bc);
    a.part_par = reinterpret_cast<float *>(ws + lo.par);
    return launched("ssd_selective_bwd", ssd::launch_sel_bwd(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_norm_fwd(const ssd_norm_dims_t *dims, const void *x, const float *weight, const float *bias, float eps,
                          void *y, float *mean, float *rstd, void *stream) {
    TRY(check_norm(dims));
    const ssd_norm_dims_t d = used(*dims);
    if (!x || !y) return fail(SSD_ERR_NULL_ARG, "x and y must be non-NULL");
    if (!(eps >= 0.f) || isinf(eps)) return fail(SSD_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels, rows = (size_t)d.rows;
    size_t nx;
    if (!span(d.rows, d.x_row_stride, 1, 0, d.channels, e, &nx))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const Tensor in[] = {{"x", x, nx, e}, {"weight", weight, ch * 4, 4}, {"bias", bias, ch * 4, 4}};
    const Tensor out[] = {{"y", y, rows * ch * e, e}, {"mean", mean, rows * 4, 4}, {"rstd", rstd, rows * 4, 4}};
    TRY(check_tensors(in, 3, out, 3));
    ssd::NormArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = d.rows;
    a.D = (int)d.channels;
    a.dtype = d.dtype;
    a.x = x;
    a.x_stride = d.x_row_stride;
    a.w = weight;
    a.bias = bias;
    a.eps = eps;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return launched("ssd_norm_fwd", ssd::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_norm_bwd_workspace_bytes(const ssd_norm_dims_t *dims) {
    return check_norm(dims) == SSD_OK ? norm_ws(*dims) : 0;
}

ssd_status_t ssd_norm_bwd(const ssd_norm_dims_t *dims, const void *dy, const void *x, const float *weight,
                          const float *mean, const float *rstd, void *dx, float *dweight, float *dbias,
                          void *workspace, size_t workspace_bytes, void *stream) {
    TRY(check_norm(dims));
    const ssd_norm_dims_t d = used(*dims);
    if (!dy || !x || !mean || !rstd || !dx) return fail(SSD_ERR_NULL_ARG, "dy, x, mean, rstd and dx must be non-NULL");
    const size_t need = norm_ws(d);
    if (!workspace || workspace_bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace %p of %zu bytes; %zu bytes are needed", workspace, workspace_bytes, need);
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels, rows = (size_t)d.rows;
    size_t nx, ng;
    if (!span(d.rows, d.x_row_stride, 1, 0, d.channels, e, &nx) || !span(d.rows, d.dy_row_stride, 1, 0, d.channels, e, &ng))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const Tensor in[] = {{"dy", dy, ng, e}, {"x", x, nx, e}, {"weight", weight, ch * 4, 4}, {"mean", mean, rows * 4, 4},
                         {"rstd", rstd, rows * 4, 4}};
    const Tensor out[] = {{"dx", dx, rows * ch * e, e}, {"dweight", dweight, ch * 4, 4}, {"dbias", dbias, ch * 4, 4},
                          {"workspace", workspace, need, 16}};
    TRY(check_tensors(in, 5, out, 4));
    ssd::NormArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = d.rows;
    a.D = (int)d.channels;
    a.dtype = d.dtype;
    a.x = x;
    a.x_stride = d.x_row_stride;
    a.dy = dy;
    a.dy_stride = d.dy_row_stride;
    a.w = weight;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.part = static_cast<float *>(workspace);
    return launched("ssd_norm_bwd", ssd::launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
