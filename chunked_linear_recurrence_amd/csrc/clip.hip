// The norm of many tensors taken together, and their clipping by it:
//
//     norm = sqrt(sum of every element's square);   out = in min(1, max_norm / norm)
//
// Two passes over the elements, the second with its writes; the norm has to be known before
// the first element is written.  Tensors are taken in batches whose pointers and sizes travel
// in the launch's arguments, so a call copies nothing to the device and can be captured.  A
// workgroup takes one chunk of one tensor.  Squares are summed in float64, in which no float32
// value's square overflows or vanishes; every workgroup of the second pass adds the chunks'
// sums in the same order, so it needs no third launch and results do not change from call to
// call.  A norm that is not finite as it is returned, in float32, changes no element.  Bound by
// memory: the second pass takes the chunks from the last to the first, which the last-level cache
// still holds: 322 MB of bfloat16 and float32 in 160 us (6.0 TB/s; in the norm's order 171), 78 of
// them for the norm.
#include "clip.h"

#include <type_traits>

namespace ssd {

// The element at which to begin with 16-byte accesses, or n where src and dst never share one
template <typename T>
__device__ __forceinline__ int64_t aligned_from(const T *src, const T *dst, int64_t n) {
    const uintptr_t a = (uintptr_t)src & 15, b = (uintptr_t)dst & 15;
    return a == b ? min((int64_t)((16 - a) % 16 / sizeof(T)), n) : n;
}

template <typename T, typename F>
__device__ __forceinline__ void each(const T *p, int64_t n, int64_t head, F f) {
    constexpr int V = 16 / (int)sizeof(T);
    for (int64_t i = threadIdx.x; i < head; i += kClipThreads) f(p + i, std::integral_constant<int, 1>{});
    const int64_t packs = (n - head) / V;
    for (int64_t i = threadIdx.x; i < packs; i += kClipThreads) f(p + head + i * V, std::integral_constant<int, V>{});
    for (int64_t i = head + packs * V + threadIdx.x; i < n; i += kClipThreads) f(p + i, std::integral_constant<int, 1>{});
}

struct ClipChunk {
    int tensor;
    int64_t first, count;
};
__device__ __forceinline__ ClipChunk clip_chunk(const ClipBatch &b, int64_t chunk, int index) {
    int lo = 0, hi = b.n;                                  // first[lo] <= index < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.first[mid] <= index) lo = mid;
        else hi = mid;
    }
    const int64_t at = (int64_t)(index - b.first[lo]) * chunk;
    return {lo, at, min(chunk, b.count(lo) - at)};
}

__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.;
#pragma unroll
    for (int w = 0; w < kClipThreads / 64; ++w) v += red[w];
    return v;
}

template <typename T>
__device__ __forceinline__ double squares(const T *p, int64_t n) {
    double s = 0.;
    each(p, n, aligned_from(p, p, n), [&](const T *q, auto width) {
        constexpr int V = decltype(width)::value;
        float v[V];
        unpack<T, V>(load_pack<T, V>(q), v);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fma((double)v[i], (double)v[i], s);
    });
    return s;
}

__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(ClipBatch b, int64_t chunk, double *part) {
    __shared__ double red[kClipThreads / 64];
    const ClipChunk c = clip_chunk(b, chunk, blockIdx.x);
    const double s = b.wide(c.tensor) ? squares(reinterpret_cast<const float *>(b.in[c.tensor]) + c.first, c.count)
                                      : squares(reinterpret_cast<const bf16 *>(b.in[c.tensor]) + c.first, c.count);
    const double sum = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// F: the factor's type.  A factor below float32's normal numbers has too few bits there, and its
// products with large elements are ordinary numbers: float64 takes it.
template <typename T, typename F>
__device__ __forceinline__ void scaled(const T *src, T *dst, int64_t n, F factor) {
    each(src, n, aligned_from(src, dst, n), [&](const T *q, auto width) {
        constexpr int V = decltype(width)::value;
        float v[V];
        unpack<T, V>(load_pack<T, V>(q), v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)(v[i] * factor);
        store_f32<T, V>(dst + (q - src), v);
    });
}

template <typename F>
__device__ __forceinline__ void scaled(const ClipBatch &b, const ClipChunk &c, F factor) {
    const void *src = b.in[c.tensor];
    void *dst = b.out[c.tensor];
    if (b.wide(c.tensor))
        scaled(reinterpret_cast<const float *>(src) + c.first, reinterpret_cast<float *>(dst) + c.first, c.count, factor);
    else
        scaled(reinterpret_cast<const bf16 *>(src) + c.first, reinterpret_cast<bf16 *>(dst) + c.first, c.count, factor);
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipBatch b, int64_t chunk, const double *part, int parts,
                                                                 double max_norm, float *norm, bool scale) {
    __shared__ double red[kClipThreads / 64];
    double s = 0.;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) s += part[i];
    const double total = sqrt(block_sum(s, red));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    if (!scale) return;
    const ClipChunk c = clip_chunk(b, chunk, gridDim.x - 1 - blockIdx.x);
    const bool clips = total > max_norm && (float)total <= 3.40282347e38f;
    if (!clips && b.in[c.tensor] == b.out[c.tensor]) return;
    const double factor = clips ? max_norm / total : 1.;
    if (factor < 0x1p-126) scaled(b, c, factor);
    else scaled(b, c, (float)factor);
}

// Elements of a chunk: about 2048 chunks in all, 4096 elements at least.
static int64_t chunk_of(const ClipArgs &a) {
    int64_t total = 0;
    for (int i = 0; i < a.n; ++i) total += a.counts[i];
    const int64_t c = (total / 2048 + 4095) / 4096 * 4096;
    return c < 4096 ? 4096 : c;
}

int64_t clip_chunks(const ClipArgs &a) {
    const int64_t chunk = chunk_of(a);
    int64_t n = 0;
    for (int i = 0; i < a.n; ++i) n += (a.counts[i] + chunk - 1) / chunk;
    return n;
}

hipError_t launch_clip(const ClipArgs &a, hipStream_t s) {
    const int64_t chunk = chunk_of(a), parts = clip_chunks(a);
    for (int pass = 0; pass < 2; ++pass) {
        int64_t at = 0;
        bool first = true;
        for (int i = 0; i < a.n || (pass == 1 && first);) {
            ClipBatch b;
            b.n = 0;
            b.first[0] = 0;
            for (; i < a.n && b.n < kClipTensors; ++i) {
                if (a.counts[i] == 0) continue;
                b.in[b.n] = a.in[i];
                b.out[b.n] = a.out ? a.out[i] : nullptr;
                b.size[b.n] = a.counts[i] * 2 + (a.dtypes[i] == SSD_F32);
                b.first[b.n + 1] = b.first[b.n] + (int)((a.counts[i] + chunk - 1) / chunk);
                ++b.n;
            }
            const int blocks = b.first[b.n];
            if (pass == 0) {
                if (blocks) clip_norm_kernel<<<blocks, kClipThreads, 0, s>>>(b, chunk, a.part + at);
            } else {
                const bool scale = a.out && blocks;
                if (scale || first)
                    clip_scale_kernel<<<scale ? blocks : 1, kClipThreads, 0, s>>>(b, chunk, a.part, (int)parts, a.max_norm,
                                                                                  first ? a.norm : nullptr, scale);
            }
            first = false;
            at += blocks;
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            if (pass == 1 && !a.out) break;
        }
    }
    return hipSuccess;
}

}  // namespace ssd
