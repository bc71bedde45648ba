// What the C entries of the operators around a scan share: their tensors' extents, alignment
// and overlaps, and the status of a launch.
#pragma once

#include <initializer_list>

#include <hip/hip_runtime.h>

#include "ssd_check.h"

namespace ssd_check {

// A tensor of a call: where it lies, its bytes, and the alignment its elements need.
struct Tensor {
    const char *name;
    const void *p;
    size_t bytes;
    uintptr_t align;
};

constexpr int64_t kMaxElems = INT64_C(1) << 58;   // spans stay far from int64 overflow in bytes

inline bool product(std::initializer_list<int64_t> f, int64_t *out) {
    int64_t r = 1;
    for (int64_t v : f)
        if (!mul_ok(r, v, kMaxElems, &r)) return false;
    *out = r;
    return true;
}

// Bytes from the first to the last element of a view [batch, seqlen, channels].
inline bool span(int64_t batch, int64_t bs, int64_t len, int64_t ts, int64_t ch, int64_t e, size_t *out) {
    int64_t a, b;
    if (bs < 0 || ts < 0 || !mul_ok(batch - 1, bs, kMaxElems, &a) || !mul_ok(len - 1, ts, kMaxElems, &b)) return false;
    *out = (size_t)(a + b + ch) * (size_t)e;
    return true;
}

inline ssd_status_t check_tensors(const Tensor *in, int nin, const Tensor *out, int nout) {
    for (int i = 0; i < nin + nout; ++i) {
        const Tensor &t = i < nin ? in[i] : out[i - nin];
        if (t.p && ((uintptr_t)t.p & (t.align - 1)))
            return fail(SSD_ERR_MISALIGNED, "%s is not %d-byte aligned", t.name, (int)t.align);
    }
    for (int o = 0; o < nout; ++o) {
        if (!out[o].p) continue;
        for (int k = 0; k < nin; ++k)
            if (in[k].p && overlap(out[o].p, out[o].bytes, in[k].p, in[k].bytes))
                return fail(SSD_ERR_ALIAS, "%s overlaps %s", out[o].name, in[k].name);
        for (int k = 0; k < o; ++k)
            if (out[k].p && overlap(out[o].p, out[o].bytes, out[k].p, out[k].bytes))
                return fail(SSD_ERR_ALIAS, "%s overlaps %s", out[o].name, out[k].name);
    }
    return SSD_OK;
}

inline ssd_status_t check_dtype(int32_t dtype) {
    if (dtype != SSD_F32 && dtype != SSD_BF16)
        return fail(SSD_ERR_BAD_DTYPE, "dtype %d is not SSD_F32 (0) or SSD_BF16 (1)", dtype);
    return SSD_OK;
}

inline ssd_status_t launched(const char *what, hipError_t e) {
    if (e == hipErrorInvalidValue)
        return fail(SSD_ERR_UNSUPPORTED, "%s: the work exceeds the grid range", what);
    if (e != hipSuccess) return fail(SSD_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace ssd_check

#define TRY(expr)                                  \
    do {                                           \
        const ssd_status_t st_ = (expr);           \
        if (st_ != SSD_OK) return st_;             \
    } while (0)
