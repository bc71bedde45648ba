/*
 * libssdscan -- chunked scan of a diagonal-decay selective state-space layer on
 * AMD Instinct MI355X (gfx950).
 *
 * The method is the one of the page
 *   "分块推理：解锁循环模型并行计算，实现长序列高效处理"
 * (chunked inference for recurrent models), cited below as [分块推理 §n].
 *
 * One layer computes, for every batch row b and head h, the recurrence of [分块推理 §2]
 *
 *     a_t = exp(dt[b,t,h] * A[h])                      (per-token, per-head decay)
 *     S_t = a_t * S_{t-1} + x[b,t,h,:] (outer) B[b,t,g,:]   (state S is P x N)
 *     y[b,t,h,p] = sum_n C[b,t,g,n] * S_t[p,n] + D[h] * x[b,t,h,p]
 *
 * with S_{-1} = init_state (or 0) and g = h / (H / G).  The library reaches this result by
 * the chunked decomposition of [分块推理 §2.1-§2.2]: split the sequence into chunks of Q
 * tokens; compute every chunk's intra output and local end state from a zero state;
 * pass the global state b(c) = b_intra(c) + (prod of a_t over chunk c) * b(c-1) across
 * chunks; and correct every chunk's output by diag(L) C b(c-1), where L_i is the product
 * of a_t from the chunk start to token i inclusive.
 *
 * Conventions (readings of the page, which leaves them open):
 *   - dt enters only through a_t; the input term is x (outer) B with no dt factor.
 *   - No softplus, bias or clamp is applied to dt; it is used as given.
 *   - D (skip term) is optional; NULL means no skip term.
 *
 * ---------------------------------------------------------------------------------
 * Memory, ownership, streams
 *   Every pointer argument is device memory owned by the caller (for example a torch
 *   tensor's data pointer).  The library never allocates or frees device memory; the
 *   caller provides a workspace of at least the size the *_workspace_bytes query returns.
 *   All work is enqueued on `stream` (a hipStream_t; NULL is the default stream) and
 *   returns without waiting.  Argument errors are detected on the host before anything
 *   is enqueued, and then nothing is written.  A fault inside a kernel surfaces at the
 *   caller's next synchronisation.  No C++ exception crosses this interface.
 *   The library holds no global mutable state except a per-thread error message (and a
 *   once-per-device kernel attribute), so concurrent calls on different workspaces are
 *   safe.  No entry point allocates or synchronises, so calls can be captured in HIP
 *   graphs.
 *
 * Layouts (row-major, contiguous, element types in parentheses; "act" = the dims' dtype)
 *   x, y             [batch, seqlen, nheads, headdim]          (act)
 *   dt               [batch, seqlen, nheads]                   (act)
 *   A, D             [nheads]                                  (float32)
 *   B, C             [batch, seqlen, ngroups, dstate]          (act)
 *   init_state,
 *   final_state      [batch, nheads, headdim, dstate]          (float32)
 *   x, y, B, C, init_state, final_state, layer_states and the workspace must be 16-byte
 *   aligned; A and D 4-byte aligned; dt aligned to its element size.
 *
 * Supported shapes on the GPU path (others return SSD_ERR_UNSUPPORTED):
 *   chunk_Q in {32, 64, 128, 256}; headdim in {16, 32, 64, 128}; dstate in {16, 32, 64, 128,
 *   256} (bfloat16 needs dstate >= 32); the set actually compiled is reported by
 *   ssd_shape_supported().  Any batch, seqlen >= 1, nheads >= 1 with nheads % ngroups == 0.
 *   The last chunk may be shorter than Q.
 *
 * Values: every a_t must be a decay, 0 <= a_t <= 1, i.e. dt >= 0 and A <= 0, both finite
 *   (as the state transition of [分块推理 §2] is in every workload).  The kernels rely on
 *   it: the log-decay prefix sums of dt * A never increase along a chunk, so every decay
 *   they form between two tokens is exp of a non-positive number (the diagonal tiles of
 *   ssd_chunk_scan_fwd clamp that exponent at 0 to mask the tokens after i).  With a
 *   growing a_t (dt * A > 0) the results are unspecified: they are wrong, and may
 *   overflow.  The library cannot check device-resident values without synchronising, so
 *   it does not; this contract applies to ssd_chunk_scan_fwd, ssd_chunk_scan_stages,
 *   ssd_chunk_scan_segmented and ssd_step.
 *
 * Tuning (environment, read at each call; optional): SSD_HEADS_PER_WG_STATE and
 *   SSD_HEADS_PER_WG_SCAN set how many heads one workgroup of chunk_state / chunk_scan
 *   processes (by default chosen from the problem size).  They change only how the work
 *   is split, never the arithmetic: results are bit-identical for every value.
 */
#ifndef LIBSSDSCAN_H
#define LIBSSDSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ssd_status {
    SSD_OK = 0,
    SSD_ERR_NULL_ARG = 1,     /* a required pointer is NULL                          */
    SSD_ERR_BAD_SHAPE = 2,    /* a dimension <= 0, nheads % ngroups != 0, V < 1, ... */
    SSD_ERR_BAD_DTYPE = 3,    /* dims.dtype is not an ssd_dtype_t value               */
    SSD_ERR_UNSUPPORTED = 4,  /* a valid shape that no compiled kernel covers         */
    SSD_ERR_MISALIGNED = 5,   /* a pointer is not 16-byte aligned                     */
    SSD_ERR_WORKSPACE = 6,    /* workspace NULL or smaller than the query's size      */
    SSD_ERR_HIP = 7,          /* a HIP launch failed (message has the HIP error)      */
    SSD_ERR_ALIAS = 8         /* an output overlaps an input it must not overlap      */
} ssd_status_t;

typedef enum ssd_dtype {
    SSD_F32 = 0,   /* activations stored and computed in float32 (fp32 matrix cores)        */
    SSD_BF16 = 1   /* activations stored in bfloat16, products on bf16 matrix cores, fp32
                      accumulation.  The state carried across chunks is summed in float32;
                      the per-chunk states stored in the workspace (b_intra, b_in) are
                      rounded to bfloat16; decays, init_state and final_state are float32 */
} ssd_dtype_t;

typedef struct ssd_dims {
    int64_t batch;     /* b                                   */
    int64_t seqlen;    /* L, tokens in this call              */
    int64_t nheads;    /* H                                   */
    int64_t headdim;   /* P, x channels per head              */
    int64_t dstate;    /* N, state size per channel           */
    int64_t ngroups;   /* G, B/C groups; head h reads group h / (H / G) */
    int32_t dtype;     /* ssd_dtype_t                         */
    int32_t reserved;  /* must be 0                           */
} ssd_dims_t;

/* flags */
#define SSD_FLAG_RESIDUAL 1u   /* y = (recurrence output + D x) + x, rounded once to act */
#define SSD_FLAG_WAVEFRONT 2u  /* segmented stack only: run independent (segment, layer)
                                  steps together (see ssd_chunk_scan_segmented) */
#define SSD_FLAG_SCAN_FORM 4u  /* ssd_chunk_scan_fwd / _stages only: compute the chunk outputs
                                  with the associative-scan form of [分块推理 §2.1] (a
                                  log-depth tree over the pairs (a_t, x_t B_t) on the vector
                                  units) instead of the matrix-core form; same results within
                                  the tolerances, for comparison.  Shapes:
                                  ssd_scan_form_supported(). */

/* Size in bytes of the workspace ssd_chunk_scan_fwd needs for these dims and chunk_Q,
 * or 0 when the arguments are invalid.  The workspace holds the per-chunk log-decay
 * prefix sums (with each chunk's total), each token's decay to the end of its 16-token
 * block (4 bytes per token and head), and two per-chunk state buffers (nheads * headdim *
 * dstate * 2 * act bytes / chunk_Q bytes per token). */
size_t ssd_chunk_scan_workspace_bytes(const ssd_dims_t *dims, int32_t chunk_Q);

/* One layer, the whole sequence [分块推理 §2-§2.2].
 *   x, dt, A, B, C     inputs (layouts above); D and init_state may be NULL.
 *   chunk_Q            chunk length Q [分块推理 §2, §4.1].
 *   y                  output [batch, seqlen, nheads, headdim] (act); must not overlap x.
 *   final_state        state after the last token, or NULL; may be the same pointer as
 *                      init_state (updated in place), no other overlap allowed.
 *   flags              0, SSD_FLAG_RESIDUAL and/or SSD_FLAG_SCAN_FORM.
 *   workspace          caller-owned device scratch; its contents on entry do not matter.
 * Returns SSD_OK once the kernels are enqueued on `stream`. */
ssd_status_t ssd_chunk_scan_fwd(const ssd_dims_t *dims, const void *x, const void *dt,
                                const float *A, const void *B, const void *C,
                                const float *D, const float *init_state, int32_t chunk_Q,
                                void *y, float *final_state, uint32_t flags,
                                void *workspace, size_t workspace_bytes, void *stream);

/* ssd_chunk_scan_fwd for callers that cannot allocate or pass device memory for a
 * workspace (code under HIP graph capture that must not allocate, tight serving loops,
 * harnesses that forbid allocation): the same computation, the same kernels and
 * bit-identical results, with the workspace taken from a scratch array inside the
 * library instead of a caller buffer.  Nothing is allocated or freed here.
 *   Arguments as for ssd_chunk_scan_fwd, without workspace and workspace_bytes.
 *   Limit: the workspace ssd_chunk_scan_workspace_bytes reports for these dims and chunk_Q
 *   must not exceed SSD_NOALLOC_SCRATCH_BYTES (64 MiB; for example up to ~41K tokens of
 *   batch * seqlen at nheads 24, headdim 64, dstate 128, chunk_Q 256, bf16); larger calls
 *   return SSD_ERR_WORKSPACE before anything is enqueued.
 *   Each GPU the library runs on holds one such array from the library's load until the
 *   process ends, shared by every call on that GPU: calls that overlap on one GPU (on
 *   different streams, or from several threads) race on it and must be serialised by
 *   the caller.  The first call on a device resolves the array's address there.
 * Returns SSD_OK once the kernels are enqueued on `stream`. */
#define SSD_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
ssd_status_t ssd_chunk_scan_fwd_noalloc(const ssd_dims_t *dims, const void *x, const void *dt,
                                        const float *A, const void *B, const void *C,
                                        const float *D, const float *init_state, int32_t chunk_Q,
                                        void *y, float *final_state, uint32_t flags, void *stream);

/* Workspace size for ssd_chunk_scan_segmented with these n_layers and flags (0 when the
 * arguments are invalid).  Without SSD_FLAG_WAVEFRONT it is two segment buffers and one
 * layer workspace over V tokens; with it, depth = min(ceil(seqlen / V), n_layers) times
 * that.  Either way it is bounded independently of seqlen: memory stays at a fixed number
 * of segments plus the caller's per-layer states, whatever the sequence length
 * [分块推理 §3.2]. */
size_t ssd_segmented_workspace_bytes(const ssd_dims_t *dims, int32_t chunk_Q, int64_t V,
                                     int32_t n_layers, uint32_t flags);

/* A stack of n_layers layers run in the vertical order of [分块推理 §3.2]: the sequence is
 * cut into segments of V tokens (the last may be shorter); each segment goes through
 * every layer before the next segment starts, and each layer's state is carried between
 * segments in layer_states.
 *   dims               shape of one layer; dims.seqlen is the full length L.
 *   x0                 stack input [batch, L, nheads, headdim] (act).
 *   dt, B, C           shared by every layer (layouts above).
 *   A, D               per layer, [n_layers, nheads] float32 (D may be NULL).
 *   layer_states       [n_layers, batch, nheads, headdim, dstate] float32, in: each layer's
 *                      initial state, out: its state after token L-1.  This is the
 *                      per-(layer) state store of [分块推理 §3.2]; copying it out and back
 *                      between calls resumes the stack exactly.
 *   y                  stack output [batch, L, nheads, headdim] (act): the last layer's
 *                      output; must not overlap x0.
 *   flags              SSD_FLAG_RESIDUAL (applied at every layer) and/or
 *                      SSD_FLAG_WAVEFRONT.
 * Layer l maps u to (recurrence_l(u) + D_l u [+ u]) rounded to act.  When V is a multiple
 * of chunk_Q the result is bit-identical to running ssd_chunk_scan_fwd layer by layer over
 * the whole sequence (the horizontal order of [分块推理 §3.1]).
 * Schedule: step (s, l) is segment s through layer l.  It needs (s, l-1) (its input) and
 * (s-1, l) (layer l's state), nothing else.  Without SSD_FLAG_WAVEFRONT the steps run one
 * at a time, segment by segment, as the page describes.  With it, all steps of one
 * anti-diagonal s + l = const run in the same four kernel launches (up to
 * min(segments, n_layers) steps at once), which fills the GPU when a single step is
 * small; every step computes exactly what it computes alone, so the output and states
 * are bit-identical between the two schedules. */
ssd_status_t ssd_chunk_scan_segmented(const ssd_dims_t *dims, int32_t n_layers, int64_t V,
                                      const void *x0, const void *dt, const float *A,
                                      const void *B, const void *C, const float *D,
                                      float *layer_states, int32_t chunk_Q, uint32_t flags,
                                      void *y, void *workspace, size_t workspace_bytes,
                                      void *stream);

/* One decode step: the next token of the recurrence of [分块推理 §2], continuing from
 * a carried state (for example the final_state of a chunked prefill), as the per-layer
 * fixed-size state of [分块推理 §2.3] is kept between tokens during generation:
 *     a = exp(dt[b,h] A[h]);   state = a state + x (outer) B;
 *     y[b,h,p] = sum_n C[b,g,n] state[b,h,p,n] + D[h] x[b,h,p]   (+ x with SSD_FLAG_RESIDUAL)
 *   dims        shape of one layer; dims.seqlen must be 1.
 *   x           [batch, nheads, headdim] (act), the token's input.
 *   dt          [batch, nheads] (act).
 *   A, D        [nheads] float32; D may be NULL.
 *   B, C        [batch, ngroups, dstate] (act).
 *   state       [batch, nheads, headdim, dstate] float32, read and written in place.
 *   y           [batch, nheads, headdim] (act); must not overlap x or state.
 *   flags       0 or SSD_FLAG_RESIDUAL.
 * dstate must be one of 16, 32, 64, 128, 256; any headdim >= 1.  Alignment: state, B and
 * C 16 bytes; x, dt, y their element size; A and D 4 bytes.  No workspace; nothing is
 * allocated.  Returns SSD_OK once the kernel is enqueued on `stream`. */
ssd_status_t ssd_step(const ssd_dims_t *dims, const void *x, const void *dt, const float *A,
                      const void *B, const void *C, const float *D, float *state, void *y,
                      uint32_t flags, void *stream);

/* ---- the operators around a scan ------------------------------------------------- *
 *
 * A selective block runs norm -> projection -> short causal convolution -> selective scan
 * (gated) -> projection; the convolution stands in front of ssd_chunk_scan_fwd as well.
 * Each operator has a forward for prompts, the convolution and the scan one for a single
 * token, and each a backward.  They share the conventions above (caller-owned device
 * memory, caller's workspace, errors before anything is enqueued, no allocation, no
 * synchronisation) with these differences:
 *
 * Strides.  An activation input may be a view: rows of contiguous channels at any
 *   batch and token stride (elements, >= 0), for example one half of a projection's output.
 *   The strides are fields of the dims; those over a dimension of one element, and those of a
 *   tensor that is not given, are not looked at.  Outputs, states and parameters are contiguous.
 * Alignment.  Pointers are aligned to their element size; B and C rows, in bfloat16, to 4
 *   bytes (even strides) except for a single token.  Where addresses and sizes allow 16-byte accesses, the
 *   convolution and the norm use them; results are the same either way.  Single-token
 *   states of the scan must be 16-byte aligned.
 * Lengths.  `lengths` (device, int32 [batch], or NULL for seqlen everywhere) gives each
 *   row's own tokens, clamped to 0..seqlen.  Tokens past a row's length are not read into
 *   any result (whatever they hold), their outputs and gradients are 0, and the final state
 *   is the one after the row's last token (the initial state of an empty row).
 * Range.  A call whose work exceeds one launch of the device (2^32 threads) is refused with
 *   SSD_ERR_UNSUPPORTED.
 * Arithmetic.  Everything is computed in float32 and rounded once when stored in the
 *   activation dtype; parameters, their gradients and the scan's states are float32.
 *   Sums over tokens, rows and channels are added in a fixed order: results do not change
 *   from call to call.
 */
#define SSD_FLAG_SILU 8u       /* ssd_conv_*: y = pre * sigmoid(pre) instead of y = pre      */
#define SSD_FLAG_SOFTPLUS 16u  /* ssd_selective_*: dt = log(1 + exp(delta + delta_bias))
                                  instead of dt = delta + delta_bias                          */

typedef struct ssd_conv_dims {
    int64_t batch, seqlen, channels;
    int32_t width;     /* W: taps, 2..4                                                  */
    int32_t dtype;     /* ssd_dtype_t                                                    */
    int64_t x_batch_stride, x_token_stride;
    int64_t dy_batch_stride, dy_token_stride;   /* backward only                         */
} ssd_conv_dims_t;

/* Short causal convolution of every channel:
 *     pre[b,t,c] = bias[c] + sum_j weight[c,j] x[b, t - (W-1) + j, c];  y = pre, or its SiLU
 *   x            view [batch, seqlen, channels] (act)
 *   weight       [channels, W] float32; bias [channels] float32 or NULL
 *   init_state   [batch, W-1, channels] (act) or NULL (zeros): the inputs before the first
 *                token, oldest first
 *   y            [batch, seqlen, channels] (act)
 *   final_state  [batch, W-1, channels] (act) or NULL: the last W-1 inputs of each row; may
 *                be init_state (updated in place)
 *   flags        0 or SSD_FLAG_SILU */
ssd_status_t ssd_conv_fwd(const ssd_conv_dims_t *dims, const void *x, const float *weight, const float *bias,
                          const void *init_state, const int32_t *lengths, void *y, void *final_state,
                          uint32_t flags, void *stream);

/* One token: dims.seqlen must be 1; x [batch, channels] at x_batch_stride, state_in and
 * state_out [batch, W-1, channels] (act; the same pointer updates in place), y [batch, channels]. */
ssd_status_t ssd_conv_step(const ssd_conv_dims_t *dims, const void *x, const float *weight, const float *bias,
                           const void *state_in, void *state_out, void *y, uint32_t flags, void *stream);

/* Gradients of ssd_conv_fwd, from dy (view, act) and dfinal ([batch, W-1, channels] (act),
 * the gradient of final_state, or NULL): dx [batch, seqlen, channels] (act), dweight
 * [channels, W] and dbias [channels] (or NULL) float32, dinit [batch, W-1, channels] (act,
 * or NULL).  The other arguments are the forward's. */
size_t ssd_conv_bwd_workspace_bytes(const ssd_conv_dims_t *dims);
ssd_status_t ssd_conv_bwd(const ssd_conv_dims_t *dims, const void *dy, const void *x, const float *weight,
                          const float *bias, const void *init_state, const void *dfinal, const int32_t *lengths,
                          void *dx, float *dweight, float *dbias, void *dinit, uint32_t flags, void *workspace,
                          size_t workspace_bytes, void *stream);

typedef struct ssd_selective_dims {
    int64_t batch, seqlen, channels;
    int64_t dstate;    /* N: 16, 32 or 64                                                */
    int64_t ngroups;   /* G: channel d reads B and C of group d / (channels / G)          */
    int32_t dtype;     /* ssd_dtype_t                                                    */
    int32_t reserved;  /* must be 0                                                      */
    int64_t u_batch_stride, u_token_stride;
    int64_t delta_batch_stride, delta_token_stride;
    int64_t z_batch_stride, z_token_stride;
    int64_t B_batch_stride, B_token_stride;
    int64_t C_batch_stride, C_token_stride;
    int64_t dy_batch_stride, dy_token_stride;   /* backward only                         */
} ssd_selective_dims_t;

/* Selective scan with a decay for every channel and state (unlike ssd_chunk_scan_fwd, the
 * input term carries dt, and dt may be derived here):
 *     dt_t = delta[b,t,d] + delta_bias[d], through SSD_FLAG_SOFTPLUS if given
 *     h_t[n] = exp(dt_t A[d,n]) h_{t-1}[n] + dt_t u[b,t,d] B[b,t,g,n]
 *     y[b,t,d] = sum_n C[b,t,g,n] h_t[n] + D[d] u[b,t,d], times z sigmoid(z) if z is given
 *   u, delta, z     views [batch, seqlen, channels] (act); z may be NULL
 *   A               [channels, dstate]; D and delta_bias [channels] or NULL (float32)
 *   B, C            views [batch, seqlen, ngroups * dstate] (act)
 *   init_state      [batch, channels, dstate] float32 or NULL (zeros)
 *   y               [batch, seqlen, channels] (act)
 *   final_state     [batch, channels, dstate] float32 or NULL; may be init_state
 *   workspace       ssd_selective_fwd_workspace_bytes (0 where enough batch rows and channels
 *                   make one pass over the sequence the faster way: it may then be NULL)
 *   kept            NULL, or ssd_selective_kept_bytes of device memory: the states before
 *                   every 8th token, which ssd_selective_bwd needs
 * Any finite A and dt whose exp(dt A) does not overflow; dt A <= 0 makes decays. */
size_t ssd_selective_kept_bytes(const ssd_selective_dims_t *dims);
size_t ssd_selective_fwd_workspace_bytes(const ssd_selective_dims_t *dims);
ssd_status_t ssd_selective_fwd(const ssd_selective_dims_t *dims, const void *u, const void *delta, const float *A,
                               const void *B, const void *C, const float *D, const void *z,
                               const float *delta_bias, const float *init_state, const int32_t *lengths, void *y,
                               float *final_state, void *kept, uint32_t flags, void *workspace,
                               size_t workspace_bytes, void *stream);

/* One token: dims.seqlen must be 1; u, delta, z and y [batch, channels], B and C [batch,
 * ngroups * dstate], at the batch strides; state_in and state_out [batch, channels, dstate]
 * float32 (the same pointer updates in place). */
ssd_status_t ssd_selective_step(const ssd_selective_dims_t *dims, const void *u, const void *delta, const float *A,
                                const void *B, const void *C, const float *D, const void *z,
                                const float *delta_bias, const float *state_in, float *state_out, void *y,
                                uint32_t flags, void *stream);

/* Gradients of ssd_selective_fwd from dy (view, act) and dfinal ([batch, channels, dstate]
 * float32, the gradient of final_state, or NULL), with the `kept` states of a forward call
 * on the same arguments.  Outputs: du, ddelta and dz [batch, seqlen, channels] (act; dz
 * exactly if z is given), dB and dC [batch, seqlen, ngroups, dstate] (act), dA [channels,
 * dstate], dD and ddelta_bias [channels] (or NULL) and dinit [batch, channels, dstate] (or
 * NULL), float32. */
size_t ssd_selective_bwd_workspace_bytes(const ssd_selective_dims_t *dims);
ssd_status_t ssd_selective_bwd(const ssd_selective_dims_t *dims, const void *dy, const void *u, const void *delta,
                               const float *A, const void *B, const void *C, const float *D, const void *z,
                               const float *delta_bias, const void *kept, const float *dfinal,
                               const int32_t *lengths, void *du, void *ddelta, float *dA, void *dB, void *dC,
                               float *dD, void *dz, float *ddelta_bias, float *dinit, uint32_t flags,
                               void *workspace, size_t workspace_bytes, void *stream);

typedef struct ssd_norm_dims {
    int64_t rows, channels;
    int32_t dtype;     /* ssd_dtype_t                                                    */
    int32_t reserved;  /* must be 0                                                      */
    int64_t x_row_stride;
    int64_t dy_row_stride;   /* backward only                                            */
} ssd_norm_dims_t;

/* Layer norm of rows of channels:
 *     y = (x - mean) rstd weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 *   x [rows, channels] (act) at x_row_stride; weight and bias [channels] float32 or NULL;
 *   eps >= 0; y [rows, channels] (act); mean and rstd [rows] float32 or NULL. */
ssd_status_t ssd_norm_fwd(const ssd_norm_dims_t *dims, const void *x, const float *weight, const float *bias,
                          float eps, void *y, float *mean, float *rstd, void *stream);

/* Gradients of ssd_norm_fwd from dy [rows, channels] (act) at dy_row_stride and the
 * forward's mean and rstd: dx [rows, channels] (act), dweight and dbias [channels] float32
 * (or NULL). */
size_t ssd_norm_bwd_workspace_bytes(const ssd_norm_dims_t *dims);
ssd_status_t ssd_norm_bwd(const ssd_norm_dims_t *dims, const void *dy, const void *x, const float *weight,
                          const float *mean, const float *rstd, void *dx, float *dweight, float *dbias,
                          void *workspace, size_t workspace_bytes, void *stream);

/* ---- inspection (tests and tools) ------------------------------------------------ */

/* Runs steps first_stage..last_stage of ssd_chunk_scan_fwd (1 = log-decay prefix sums,
 * 2 = per-chunk local states, 3 = state pass, 4 = chunk outputs) and leaves the
 * intermediates in the workspace (see ssd_workspace_layout).  A step reads what the
 * earlier steps left in the same workspace, so running 1..k and then k+1..4 with the same
 * arguments equals one ssd_chunk_scan_fwd call; running one step at a time is how each
 * kernel is timed on its own. */
ssd_status_t ssd_chunk_scan_stages(const ssd_dims_t *dims, const void *x, const void *dt,
                                   const float *A, const void *B, const void *C,
                                   const float *D, const float *init_state, int32_t chunk_Q,
                                   void *y, float *final_state, uint32_t flags,
                                   void *workspace, size_t workspace_bytes, void *stream,
                                   int32_t first_stage, int32_t last_stage);

/* Byte offsets of the intermediates inside the workspace:
 *   offsets[0]  dA_cum   [batch, nheads, nchunks, chunk_Q], float64 for SSD_F32 and float32
 *               for SSD_BF16 activations: sum of dt*A / ln 2 (the base-2 logarithm of the
 *               decay) from the chunk start to each token, inclusive (past a short last
 *               chunk: the chunk total);
 *   offsets[1]  b_intra  act dtype, per (batch, chunk, head) a P x N state in tile order;
 *   offsets[2]  b_in     act dtype, the state entering each chunk, same tile order;
 *   offsets[3]  total workspace bytes.
 * Tile order of one P x N state: 16x16 tiles indexed [n / 16][p / 16], each tile 64 lanes
 * x 4 values, where lane l, value r holds (p = 16 * (p / 16) + l % 16,
 * n = 16 * (n / 16) + 4 * (l / 16) + r). */
ssd_status_t ssd_workspace_layout(const ssd_dims_t *dims, int32_t chunk_Q, size_t offsets[4]);

/* 1 when the SSD_FLAG_SCAN_FORM kernel is compiled for (dtype, chunk_Q, headdim, dstate). */
int32_t ssd_scan_form_supported(int32_t dtype, int32_t chunk_Q, int64_t headdim, int64_t dstate);

/* 1 when a compiled kernel set covers (dtype, chunk_Q, headdim, dstate), else 0. */
int32_t ssd_shape_supported(int32_t dtype, int32_t chunk_Q, int64_t headdim, int64_t dstate);

const char *ssd_status_string(ssd_status_t status);
/* Detail of the calling thread's last error ("" when the last call succeeded). */
const char *ssd_last_error_message(void);
/* Library version: major * 10000 + minor * 100 + patch. */
int32_t ssd_version(void);

#ifdef __cplusplus
}
#endif
#endif /* LIBSSDSCAN_H */
