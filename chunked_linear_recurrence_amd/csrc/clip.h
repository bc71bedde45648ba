// Arguments and launch functions of the norm over many tensors and of clipping.
#pragma once

#include "ssd_block.h"

namespace ssd {

constexpr int kClipThreads = 512;
constexpr int kClipTensors = 128;      // of one launch: 3.6 KB of arguments, below the 4 KB there are

struct ClipBatch {
    int n;
    int first[kClipTensors + 1];       // the first chunk of each
    int64_t size[kClipTensors];        // 2 x elements, + 1 for float32
    const void *in[kClipTensors];
    void *out[kClipTensors];
    __device__ __forceinline__ int64_t count(int i) const { return size[i] >> 1; }
    __device__ __forceinline__ bool wide(int i) const { return size[i] & 1; }
};
static_assert(sizeof(ClipBatch) <= 3800, "with the other arguments within 4 KB");

struct ClipArgs {
    int n;
    const void *const *in;
    void *const *out;                  // or null: the norm alone
    const int64_t *counts;
    const int32_t *dtypes;
    double max_norm;
    float *norm;
    double *part;                      // workspace: [clip_chunks]
};

int64_t clip_chunks(const ClipArgs &a);
hipError_t launch_clip(const ClipArgs &a, hipStream_t s);

}  // namespace ssd
