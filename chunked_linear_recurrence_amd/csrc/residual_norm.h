// Arguments and launch functions of the norms around a residual.
#pragma once

#include "ssd_rows.h"

namespace ssd {

struct ResidualNormArgs {
    int64_t rows;
    int D, dtype;
    const void *branch, *gate, *residual;         // [rows, D] at their strides; gate, residual or null
    int64_t branch_stride, gate_stride, residual_stride;
    const float *post, *scale, *pre;              // [D] or null
    float eps;
    void *total, *y;                              // [rows, D]; y null without pre
    float *stats;                                 // [2, rows]: 1 / rms of t and of s; or null in the forward
    // backward
    const void *dy, *dtotal;                      // [rows, D] at their strides; dy null without pre
    int64_t dy_stride, dtotal_stride;
    void *dbranch, *dgate, *dresidual;            // dgate with gate; dresidual or null
    float *dpost, *dscale, *dpre;                 // [D] or null
    float *part;                                  // workspace: [residual_norm_bwd_blocks, 3, D]
    float *mean;                                  // workspace: [residual_norm_mean_rows]
};

bool residual_norm_fits(const ResidualNormArgs &a);
int64_t residual_norm_bwd_blocks(int64_t rows);
size_t residual_norm_mean_rows(int64_t rows, int64_t D, int dtype);
hipError_t launch_residual_norm_fwd(const ResidualNormArgs &a, hipStream_t s);
hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, hipStream_t s);

}  // namespace ssd
