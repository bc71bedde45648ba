// Host-side argument checking shared by the C-ABI entry points: the calling thread's error
// message, size arithmetic, alignment and overlap tests.
#pragma once

#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "libssdscan.h"

namespace ssd_check {

// A fixed buffer, so that recording an error can neither allocate nor throw.
inline thread_local char g_err[512] = "";

inline ssd_status_t fail(ssd_status_t st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return st;
}

inline ssd_status_t ok() {
    g_err[0] = 0;
    return SSD_OK;
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline int64_t act_bytes(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

inline bool mul_ok(int64_t a, int64_t b, int64_t lim, int64_t *out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > lim / a) return false;
    *out = a * b;
    return true;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

}  // namespace ssd_check
