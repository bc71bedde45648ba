// C-ABI entry points of a layer's feed-forward half and of its training step: the matrix
// product with its epilogue, the gated product, the norms around a residual, and clipping.
// Argument checks, workspace carving and launches on the caller's stream; nothing here
// allocates device memory or waits on the device.
#include "libssdscan.h"

#include <algorithm>

#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "clip.h"
#include "product.h"
#include "residual_norm.h"
#include "ssd_entry.h"

using namespace ssd_check;

namespace {

// ---------------------------------------------------------------------------- products
// The dims with the strides over one row, which nothing uses, as 0.
ssd_product_dims_t used(ssd_product_dims_t d) {
    if (d.rows == 1) d.x_row_stride = d.residual_row_stride = d.dy_row_stride = 0;
    return d;
}

ssd_status_t check_product(const ssd_product_dims_t *d, bool gated) {
    if (!d) return fail(SSD_ERR_NULL_ARG, "dims is NULL");
    TRY(check_dtype(d->dtype));
    if (d->reserved != 0) return fail(SSD_ERR_BAD_SHAPE, "dims.reserved must be 0");
    if (d->rows <= 0 || d->inner <= 0 || d->outer <= 0)
        return fail(SSD_ERR_BAD_SHAPE, "every dimension must be >= 1 (rows %lld inner %lld outer %lld)",
                    (long long)d->rows, (long long)d->inner, (long long)d->outer);
    if (d->rows > INT32_MAX / 2 || d->inner > INT32_MAX / 16 || d->outer > INT32_MAX / 16)
        return fail(SSD_ERR_UNSUPPORTED, "rows, inner or outer exceed the kernels' index range");
    int64_t n;
    // every tensor and workspace, the partial results of a product whose K is cut among them
    if (!product({d->rows, d->outer, gated ? 2 : 1, 512}, &n) || !product({d->outer, d->inner, gated ? 2 : 1, 512}, &n) ||
        !product({d->rows, d->inner, 512}, &n))
        return fail(SSD_ERR_BAD_SHAPE, "sizes overflow");
    return SSD_OK;
}

ssd_status_t act_of(uint32_t flags, bool gated, int *act) {
    if (flags & ~(SSD_FLAG_SILU | SSD_FLAG_GELU | SSD_FLAG_PRE_F32)) return fail(SSD_ERR_BAD_SHAPE, "unknown flags 0x%x", flags);
    const uint32_t which = flags & (SSD_FLAG_SILU | SSD_FLAG_GELU);
    if (which == (SSD_FLAG_SILU | SSD_FLAG_GELU)) return fail(SSD_ERR_BAD_SHAPE, "two activations (flags 0x%x)", flags);
    if (gated && !which) return fail(SSD_ERR_BAD_SHAPE, "a gated product has an activation (flags 0x%x)", flags);
    *act = flags & SSD_FLAG_SILU ? ssd::kActSilu : flags & SSD_FLAG_GELU ? ssd::kActGelu : ssd::kActNone;
    return SSD_OK;
}

// Bytes of an element of pre
size_t pre_bytes(int32_t dtype, uint32_t flags) { return flags & SSD_FLAG_PRE_F32 ? 4 : (size_t)act_bytes(dtype); }

ssd::ProductArgs product_args(const ssd_product_dims_t &d, bool gated) {
    ssd::ProductArgs a;
    memset(&a, 0, sizeof(a));
    a.M = d.rows;
    a.N = d.outer;
    a.K = d.inner;
    a.dtype = d.dtype;
    a.kind = gated ? ssd::kGated : ssd::kLinear;
    a.a.ld = d.x_row_stride;
    a.b.ld = d.inner;
    return a;
}

// The gradients' products over dpre [rows, cols]: by x, dpre [rows, cols] x weight [cols, inner],
// and by the weight, dpre^T [cols, rows] x x [rows, inner].
ssd::ProductArgs grad_x_args(const ssd_product_dims_t &d, int64_t cols, const void *dpre, int64_t ld, const void *weight) {
    ssd::ProductArgs a;
    memset(&a, 0, sizeof(a));
    a.M = d.rows;
    a.N = d.inner;
    a.K = cols;
    a.dtype = d.dtype;
    a.kind = ssd::kPlain;
    a.b_rows = true;
    a.a = {dpre, ld, 0};
    a.b = {weight, d.inner, 0};
    return a;
}
ssd::ProductArgs grad_w_args(const ssd_product_dims_t &d, int64_t cols, const void *dpre, int64_t ld, const void *x) {
    ssd::ProductArgs a;
    memset(&a, 0, sizeof(a));
    a.M = cols;
    a.N = d.inner;
    a.K = d.rows;
    a.dtype = d.dtype;
    a.kind = ssd::kPlain;
    a.a_rows = a.b_rows = true;
    a.a = {dpre, ld, 0};
    a.b = {x, d.x_row_stride, 0};
    return a;
}

// A backward's workspace: dpre where it is formed, the bias' partial sums, and what the two
// products need.
struct GradLayout {
    size_t dpre, sums, part, total;
};
GradLayout grad_layout(const ssd_product_dims_t &d, bool gated, bool forms) {
    const int64_t cols = gated ? 2 * d.outer : d.outer;
    GradLayout lo;
    size_t off = 0;
    lo.dpre = off;
    if (forms) off += align_up((size_t)(d.rows * cols * act_bytes(d.dtype)));
    lo.sums = off;
    off += align_up((size_t)(ssd::product_act_rows(d.rows, d.outer, d.dtype) * cols * 4));
    lo.part = off;
    const int64_t ld = forms ? cols : d.dy_row_stride;
    off += align_up(ssd::product_grads_workspace_bytes(grad_x_args(d, cols, nullptr, ld, nullptr),
                                                       grad_w_args(d, cols, nullptr, ld, nullptr)));
    lo.total = off;
    return lo;
}

size_t fwd_workspace(const ssd_product_dims_t *dims, bool gated) {
    if (check_product(dims, gated) != SSD_OK) return 0;
    return align_up(ssd::product_workspace_bytes(product_args(used(*dims), gated)));
}

ssd_status_t check_workspace(const void *p, size_t bytes, size_t need) {
    if (need && (!p || bytes < need))
        return fail(SSD_ERR_WORKSPACE, "workspace %p of %zu bytes; %zu bytes are needed", p, bytes, need);
    return SSD_OK;
}

ssd_status_t beyond(const char *what) { return fail(SSD_ERR_UNSUPPORTED, "%s: the work exceeds the grid range", what); }

ssd_status_t product_fwd(const char *what, bool gated, const ssd_product_dims_t *dims, const void *x, const void *weight,
                         const void *bias, const void *residual, void *y, void *pre, uint32_t flags, void *workspace,
                         size_t workspace_bytes, void *stream) {
    TRY(check_product(dims, gated));
    const ssd_product_dims_t d = used(*dims);
    int act;
    TRY(act_of(flags, gated, &act));
    if (!x || !weight || !y) return fail(SSD_ERR_NULL_ARG, "x, weight and %s must be non-NULL", gated ? "h" : "y");
    ssd::ProductArgs a = product_args(d, gated);
    if (!ssd::product_fits(a)) return beyond(what);
    const size_t need = align_up(ssd::product_workspace_bytes(a));
    TRY(check_workspace(workspace, workspace_bytes, need));
    const size_t e = (size_t)act_bytes(d.dtype), ep = pre_bytes(d.dtype, flags), n = (size_t)d.outer * (gated ? 2 : 1), m = (size_t)d.rows;
    size_t nx, nr = 0;
    if (!span(d.rows, d.x_row_stride, 1, 0, d.inner, (int64_t)e, &nx) ||
        (residual && !span(d.rows, d.residual_row_stride, 1, 0, d.outer, (int64_t)e, &nr)))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const Tensor in[] = {{"x", x, nx, e}, {"weight", weight, n * (size_t)d.inner * e, e}, {"bias", bias, n * e, e},
                         {"residual", residual, nr, e}};
    const Tensor out[] = {{gated ? "h" : "y", y, m * (size_t)d.outer * e, e}, {"pre", pre, m * n * ep, ep},
                          {"workspace", need ? workspace : nullptr, need, 16}};
    TRY(check_tensors(in, 4, out, 3));
    a.a.p = x;
    a.b.p = weight;
    a.bias = bias;
    a.residual = residual;
    a.residual_ld = d.residual_row_stride;
    a.act = act;
    a.y = y;
    a.pre = pre;
    a.pre_f32 = ep == 4;
    a.part = static_cast<float *>(workspace);
    return launched(what, ssd::launch_product(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t product_bwd(const char *what, bool gated, const ssd_product_dims_t *dims, const void *dy, const void *x,
                         const void *weight, const void *pre, void *dx, void *dweight, void *dbias, uint32_t flags,
                         void *workspace, size_t workspace_bytes, void *stream) {
    TRY(check_product(dims, gated));
    const ssd_product_dims_t d = used(*dims);
    int act;
    TRY(act_of(flags, gated, &act));
    const bool forms = gated || act != ssd::kActNone;         // dpre is not dy itself
    if (!dy || !x || !weight || (forms && !pre))
        return fail(SSD_ERR_NULL_ARG, "%s, x, weight%s must be non-NULL", gated ? "dh" : "dy", forms ? " and pre" : "");
    if (!forms) pre = nullptr;
    if (!dx && !dweight && !dbias) return fail(SSD_ERR_NULL_ARG, "dx, dweight and dbias are all NULL");
    const GradLayout lo = grad_layout(d, gated, forms);
    TRY(check_workspace(workspace, workspace_bytes, lo.total));
    const size_t e = (size_t)act_bytes(d.dtype), ep = pre_bytes(d.dtype, flags), m = (size_t)d.rows;
    const int64_t cols = gated ? 2 * d.outer : d.outer;
    const size_t n = (size_t)cols, k = (size_t)d.inner;
    size_t nx, ng;
    if (!span(d.rows, d.x_row_stride, 1, 0, d.inner, (int64_t)e, &nx) ||
        !span(d.rows, d.dy_row_stride, 1, 0, d.outer, (int64_t)e, &ng))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const Tensor in[] = {{gated ? "dh" : "dy", dy, ng, e}, {"x", x, nx, e}, {"weight", weight, n * k * e, e},
                         {"pre", pre, m * n * ep, ep}};
    const Tensor out[] = {{"dx", dx, m * k * e, e}, {"dweight", dweight, n * k * e, e}, {"dbias", dbias, n * e, e},
                          {"workspace", workspace, lo.total, 16}};
    TRY(check_tensors(in, 4, out, 4));
    char *ws = static_cast<char *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ssd::ProductActArgs f;
    memset(&f, 0, sizeof(f));
    f.M = d.rows;
    f.N = d.outer;
    f.dtype = d.dtype;
    f.gated = gated;
    f.dy = dy;
    f.dy_ld = d.dy_row_stride;
    f.pre = pre;
    f.pre_f32 = ep == 4;
    f.act = act;
    f.dpre = forms ? ws + lo.dpre : nullptr;
    f.part = dbias ? reinterpret_cast<float *>(ws + lo.sums) : nullptr;
    f.dbias = dbias;
    const void *dpre = forms ? f.dpre : dy;
    const int64_t ld = forms ? cols : d.dy_row_stride;
    ssd::ProductArgs gx = grad_x_args(d, cols, dpre, ld, weight), gw = grad_w_args(d, cols, dpre, ld, x);
    if (!ssd::product_act_fits(f) || !ssd::product_fits(gx) || !ssd::product_fits(gw)) return beyond(what);
    hipError_t r = hipSuccess;
    if (forms || dbias) r = ssd::launch_product_act(f, s);
    gx.y = dx;
    gw.y = dweight;
    gx.part = gw.part = reinterpret_cast<float *>(ws + lo.part);
    if (r == hipSuccess) r = ssd::launch_product_grads(gx, gw, s);
    return launched(what, r);
}

// ----------------------------------------------------------------- norms around a residual
ssd_residual_norm_dims_t used(ssd_residual_norm_dims_t d) {
    if (d.rows == 1)
        d.branch_row_stride = d.residual_row_stride = d.gate_row_stride = d.dy_row_stride = d.dtotal_row_stride = 0;
    return d;
}

ssd_status_t check_residual_norm(const ssd_residual_norm_dims_t *d) {
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

ssd::ResidualNormArgs residual_norm_args(const ssd_residual_norm_dims_t &d, const void *branch, const void *residual,
                                         const void *gate, const float *post, const float *scale, const float *pre) {
    ssd::ResidualNormArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = d.rows;
    a.D = (int)d.channels;
    a.dtype = d.dtype;
    a.branch = branch;
    a.gate = gate;
    a.residual = residual;
    a.branch_stride = d.branch_row_stride;
    a.gate_stride = gate ? d.gate_row_stride : 0;
    a.residual_stride = residual ? d.residual_row_stride : 0;
    a.post = post;
    a.scale = scale;
    a.pre = pre;
    return a;
}

// Bytes of a view of the call, 0 where it is not given.
bool view_span(const ssd_residual_norm_dims_t &d, const void *p, int64_t stride, size_t *out) {
    *out = 0;
    return !p || span(d.rows, stride, 1, 0, d.channels, act_bytes(d.dtype), out);
}

struct NormLayout {
    size_t mean, total;
};
NormLayout norm_layout(const ssd_residual_norm_dims_t &d) {
    NormLayout lo;
    lo.mean = align_up((size_t)ssd::residual_norm_bwd_blocks(d.rows) * 3 * (size_t)d.channels * 4);
    lo.total = lo.mean + align_up(ssd::residual_norm_mean_rows(d.rows, d.channels, d.dtype) * 4);
    return lo;
}

// ------------------------------------------------------------------------------- clipping
ssd_status_t check_sizes(int32_t count, const int64_t *sizes) {
    if (count < 1) return fail(SSD_ERR_BAD_SHAPE, "count must be >= 1 (got %d)", count);
    if (!sizes) return fail(SSD_ERR_NULL_ARG, "sizes is NULL");
    int64_t total = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > kMaxElems - total)
            return fail(SSD_ERR_BAD_SHAPE, "size %lld of tensor %d is negative or too large", (long long)sizes[i], i);
        total += sizes[i];
    }
    return SSD_OK;
}

ssd::ClipArgs clip_args(int32_t count, const int64_t *sizes) {
    ssd::ClipArgs a;
    memset(&a, 0, sizeof(a));
    a.n = count;
    a.counts = sizes;
    return a;
}

// A range of memory that a call reads or writes.  A tensor clipped in place is one that is written.
struct Range {
    uintptr_t from, to;
    int32_t tensor;
    bool written;
};

// No range that is written overlaps another: in the order of their starts, a range meets the
// furthest end of those before it, and that of those written.
ssd_status_t check_ranges(Range *r, int64_t n) {
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.from < b.from; });
    uintptr_t end = 0, written = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].from < written || (r[i].written && r[i].from < end))
            return fail(SSD_ERR_ALIAS, "tensor %d overlaps another that is written", r[i].tensor);
        end = std::max(end, r[i].to);
        if (r[i].written) written = std::max(written, r[i].to);
    }
    return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_linear_fwd_workspace_bytes(const ssd_product_dims_t *dims) { return fwd_workspace(dims, false); }

ssd_status_t ssd_linear_fwd(const ssd_product_dims_t *dims, const void *x, const void *weight, const void *bias,
                            const void *residual, void *y, void *pre, uint32_t flags, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return product_fwd("ssd_linear_fwd", false, dims, x, weight, bias, residual, y, pre, flags, workspace,
                       workspace_bytes, stream);
}

size_t ssd_linear_bwd_workspace_bytes(const ssd_product_dims_t *dims, uint32_t flags) {
    int act;
    if (check_product(dims, false) != SSD_OK || act_of(flags, false, &act) != SSD_OK) return 0;
    return grad_layout(used(*dims), false, act != ssd::kActNone).total;
}

ssd_status_t ssd_linear_bwd(const ssd_product_dims_t *dims, const void *dy, const void *x, const void *weight,
                            const void *pre, void *dx, void *dweight, void *dbias, uint32_t flags, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return product_bwd("ssd_linear_bwd", false, dims, dy, x, weight, pre, dx, dweight, dbias, flags, workspace,
                       workspace_bytes, stream);
}

size_t ssd_gated_fwd_workspace_bytes(const ssd_product_dims_t *dims) { return fwd_workspace(dims, true); }

ssd_status_t ssd_gated_fwd(const ssd_product_dims_t *dims, const void *x, const void *weight, const void *bias, void *h,
                           void *pre, uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
    return product_fwd("ssd_gated_fwd", true, dims, x, weight, bias, nullptr, h, pre, flags, workspace, workspace_bytes,
                       stream);
}

size_t ssd_gated_bwd_workspace_bytes(const ssd_product_dims_t *dims) {
    return check_product(dims, true) == SSD_OK ? grad_layout(used(*dims), true, true).total : 0;
}

ssd_status_t ssd_gated_bwd(const ssd_product_dims_t *dims, const void *dh, const void *x, const void *weight,
                           const void *pre, void *dx, void *dweight, void *dbias, uint32_t flags, void *workspace,
                           size_t workspace_bytes, void *stream) {
    return product_bwd("ssd_gated_bwd", true, dims, dh, x, weight, pre, dx, dweight, dbias, flags, workspace,
                       workspace_bytes, stream);
}

ssd_status_t ssd_residual_norm_fwd(const ssd_residual_norm_dims_t *dims, const void *branch, const void *residual,
                                   const void *gate, const float *post_weight, const float *scale,
                                   const float *pre_weight, float eps, void *total, void *y, float *stats,
                                   void *stream) {
    TRY(check_residual_norm(dims));
    const ssd_residual_norm_dims_t d = used(*dims);
    if (!branch || !total) return fail(SSD_ERR_NULL_ARG, "branch and total must be non-NULL");
    if (!pre_weight != !y) return fail(SSD_ERR_NULL_ARG, "y has to be given exactly if pre_weight is");
    if (!(eps >= 0.f) || isinf(eps)) return fail(SSD_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    size_t nb, nr, nz;
    if (!view_span(d, branch, d.branch_row_stride, &nb) || !view_span(d, residual, d.residual_row_stride, &nr) ||
        !view_span(d, gate, d.gate_row_stride, &nz))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels, n = (size_t)d.rows * ch * e;
    // total in place of residual: the same rows, each read before it is written
    const bool in_place = total == residual && (d.rows == 1 || d.residual_row_stride == d.channels);
    const Tensor in[] = {{"branch", branch, nb, e}, {"residual", in_place ? nullptr : residual, nr, e}, {"gate", gate, nz, e},
                         {"post_weight", post_weight, ch * 4, 4}, {"scale", scale, ch * 4, 4},
                         {"pre_weight", pre_weight, ch * 4, 4}};
    const Tensor out[] = {{"total", total, n, e}, {"y", y, n, e}, {"stats", stats, (size_t)d.rows * 8, 4}};
    TRY(check_tensors(in, 6, out, 3));
    ssd::ResidualNormArgs a = residual_norm_args(d, branch, residual, gate, post_weight, scale, pre_weight);
    a.eps = eps;
    a.total = total;
    a.y = y;
    a.stats = stats;
    if (!ssd::residual_norm_fits(a)) return beyond("ssd_residual_norm_fwd");
    return launched("ssd_residual_norm_fwd", ssd::launch_residual_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_residual_norm_bwd_workspace_bytes(const ssd_residual_norm_dims_t *dims) {
    return check_residual_norm(dims) == SSD_OK ? norm_layout(*dims).total : 0;
}

ssd_status_t ssd_residual_norm_bwd(const ssd_residual_norm_dims_t *dims, const void *dy, const void *dtotal,
                                   const void *branch, const void *residual, const void *gate,
                                   const float *post_weight, const float *scale, const float *pre_weight,
                                   const float *stats, void *dbranch, void *dresidual, void *dgate,
                                   float *dpost_weight, float *dscale, float *dpre_weight, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    TRY(check_residual_norm(dims));
    const ssd_residual_norm_dims_t d = used(*dims);
    if (!branch || !stats || !dbranch) return fail(SSD_ERR_NULL_ARG, "branch, stats and dbranch must be non-NULL");
    if (!pre_weight != !dy) return fail(SSD_ERR_NULL_ARG, "dy has to be given exactly if pre_weight is");
    if (!dy && !dtotal) return fail(SSD_ERR_NULL_ARG, "dy and dtotal are both NULL");
    if (!gate != !dgate) return fail(SSD_ERR_NULL_ARG, "dgate has to be given exactly if gate is");
    if ((dresidual && !residual) || (dpost_weight && !post_weight) || (dscale && !scale) || (dpre_weight && !pre_weight))
        return fail(SSD_ERR_NULL_ARG, "a gradient is given whose input is not");
    const NormLayout lo = norm_layout(d);
    TRY(check_workspace(workspace, workspace_bytes, lo.total));
    size_t nb, nr, nz, ng, nt;
    if (!view_span(d, branch, d.branch_row_stride, &nb) || !view_span(d, residual, d.residual_row_stride, &nr) ||
        !view_span(d, gate, d.gate_row_stride, &nz) || !view_span(d, dy, d.dy_row_stride, &ng) ||
        !view_span(d, dtotal, d.dtotal_row_stride, &nt))
        return fail(SSD_ERR_BAD_SHAPE, "strides must be >= 0 and spans below 2^58 elements");
    const size_t e = (size_t)act_bytes(d.dtype), ch = (size_t)d.channels, n = (size_t)d.rows * ch * e;
    const Tensor in[] = {{"dy", dy, ng, e}, {"dtotal", dtotal, nt, e}, {"branch", branch, nb, e},
                         {"residual", residual, nr, e}, {"gate", gate, nz, e}, {"post_weight", post_weight, ch * 4, 4},
                         {"scale", scale, ch * 4, 4}, {"pre_weight", pre_weight, ch * 4, 4},
                         {"stats", stats, (size_t)d.rows * 8, 4}};
    const Tensor out[] = {{"dbranch", dbranch, n, e}, {"dresidual", dresidual, n, e}, {"dgate", dgate, n, e},
                          {"dpost_weight", dpost_weight, ch * 4, 4}, {"dscale", dscale, ch * 4, 4},
                          {"dpre_weight", dpre_weight, ch * 4, 4}, {"workspace", workspace, lo.total, 16}};
    TRY(check_tensors(in, 9, out, 7));
    ssd::ResidualNormArgs a = residual_norm_args(d, branch, residual, gate, post_weight, scale, pre_weight);
    a.stats = const_cast<float *>(stats);
    a.dy = dy;
    a.dtotal = dtotal;
    a.dy_stride = dy ? d.dy_row_stride : 0;
    a.dtotal_stride = dtotal ? d.dtotal_row_stride : 0;
    a.dbranch = dbranch;
    a.dresidual = dresidual;
    a.dgate = dgate;
    a.dpost = dpost_weight;
    a.dscale = dscale;
    a.dpre = dpre_weight;
    a.part = static_cast<float *>(workspace);
    a.mean = reinterpret_cast<float *>(static_cast<char *>(workspace) + lo.mean);
    if (!ssd::residual_norm_fits(a)) return beyond("ssd_residual_norm_bwd");
    return launched("ssd_residual_norm_bwd", ssd::launch_residual_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_clip_workspace_bytes(int32_t count, const int64_t *sizes) {
    if (check_sizes(count, sizes) != SSD_OK) return 0;
    return align_up((size_t)ssd::clip_chunks(clip_args(count, sizes)) * 8 + 8);
}

ssd_status_t ssd_clip(int32_t count, const void *const *in, void *const *out, const int64_t *sizes,
                      const int32_t *dtypes, double max_norm, float *norm, void *workspace, size_t workspace_bytes,
                      void *stream) {
    TRY(check_sizes(count, sizes));
    if (!in || !dtypes || !norm) return fail(SSD_ERR_NULL_ARG, "in, dtypes and norm must be non-NULL");
    if (out && !(max_norm >= 0.)) return fail(SSD_ERR_BAD_SHAPE, "max_norm must be >= 0");
    const size_t need = ssd_clip_workspace_bytes(count, sizes);
    TRY(check_workspace(workspace, workspace_bytes, need));
    for (int32_t i = 0; i < count; ++i) {
        TRY(check_dtype(dtypes[i]));
        if (sizes[i] == 0) continue;
        if (!in[i] || (out && !out[i])) return fail(SSD_ERR_NULL_ARG, "tensor %d is NULL", i);
        const uintptr_t e = (uintptr_t)act_bytes(dtypes[i]) - 1;
        if (((uintptr_t)in[i] & e) || (out && ((uintptr_t)out[i] & e)))
            return fail(SSD_ERR_MISALIGNED, "tensor %d is not aligned to its elements", i);
    }
    if (((uintptr_t)norm & 3u) || ((uintptr_t)workspace & 15u))
        return fail(SSD_ERR_MISALIGNED, "norm is not 4-byte aligned or workspace not 16-byte aligned");
    Range *ranges = static_cast<Range *>(malloc(sizeof(Range) * (2 * (size_t)count + 2)));
    if (!ranges) return fail(SSD_ERR_WORKSPACE, "no host memory for the check of %d tensors", count);
    int64_t n = 0;
    auto add = [&](const void *p, size_t bytes, int32_t i, bool written) {
        ranges[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, i, written};
    };
    for (int32_t i = 0; i < count; ++i) {
        const size_t bytes = (size_t)sizes[i] * (size_t)act_bytes(dtypes[i]);
        if (!bytes) continue;
        if (!out || out[i] != in[i]) add(in[i], bytes, i, false);
        if (out) add(out[i], bytes, i, true);
    }
    add(norm, 4, count, true);
    add(workspace, need, count, true);
    const ssd_status_t st = check_ranges(ranges, n);
    free(ranges);
    if (st != SSD_OK) return st;
    ssd::ClipArgs a = clip_args(count, sizes);
    a.in = in;
    a.out = out;
    a.dtypes = dtypes;
    a.max_norm = max_norm;
    a.norm = norm;
    a.part = static_cast<double *>(workspace);
    return launched("ssd_clip", ssd::launch_clip(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
