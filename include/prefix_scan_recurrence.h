/*
 * prefix_scan_recurrence.h -- C ABI of the gated linear recurrence: the scan of
 * affine maps (ps_scan_affine_f32) that a recurrent layer runs over its tokens,
 * channel by channel,
 *
 *     h_t = exp(g_t) h_{t-1} + w_t x_t
 *
 * with an input x, a log decay g and a state h of one number each for every
 * channel of every token.  w is 1, or, where input and decay are tied,
 * 1 - exp(g).  (The gated delta rule, prefix_scan_delta.h, is the same with
 * matrices as states.)
 *
 * Types: x, h and their gradients are of one type (f32, bf16 or f16), g and its
 * gradient of that type or f32; states, their gradients and all sums are f32.
 * Results repeat bit for bit from call to call.  A token's factor exp(g) is off by
 * 2^-21.5 at most, and near 1 (g > -1/16) by 2^-22.3 of its distance from 1, so that
 * errors do not add up over long memories; the weight 1 - exp(g) is off by 2^-20.2
 * of itself at most for x of f32, by 2^-18.7 for x of 16 bits.
 *
 * Log decays are at most 0 as a rule.  Above 0 states grow; sums of g over 512
 * tokens then have to stay below 80.  -infinity forgets the state: what follows
 * does not depend on it, unless it was not finite.  NaN and infinities reach the
 * channel's later outputs in their own sequence (and earlier tokens' gradients),
 * and no others; an infinity may go on as NaN.
 *
 * A kernel whose bounded waits ran out, which a correct launch never does,
 * finishes instead of hanging, with NaN in the outputs that rest on what it
 * waited for.
 *
 * Conventions: device pointers owned by the caller; work is enqueued on
 * `stream` and the call returns without waiting for it; no device memory is
 * allocated and nothing is kept between calls; calls can be captured in CUDA
 * graphs.  Errors found on the host are returned before anything is enqueued:
 * PS_ERR_INVALID_ARG (a bad enum, size, stride or pointer),
 * PS_ERR_WORKSPACE_TOO_SMALL, PS_ERR_OVERLAP (an output that meets an input,
 * another output or the workspace), PS_ERR_CUDA.  The workspace needs no
 * preparation; calls that may run at the same time must not share one.
 */
#ifndef PREFIX_SCAN_RECURRENCE_H
#define PREFIX_SCAN_RECURRENCE_H

#include "prefix_scan_delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A tensor over (sequence, token, channel): strides in elements; channels are
 * contiguous.  For packed sequences the token index runs over all of them and
 * seq_stride is not used.  Stride 0 (a broadcast input) is fine.
 */
typedef struct ps_linrec_tensor {
    const void *data;
    int64_t seq_stride;
    int64_t tok_stride;
} ps_linrec_tensor;

/*
 * num_seqs   sequences (0: nothing to do)
 * tokens     tokens of every sequence; with cu_seqlens, of all together
 * cu_seqlens NULL, or a device array of num_seqs + 1 offsets: sequence i has
 *            tokens [cu[i], cu[i+1]).  Offsets are read on the device and
 *            clamped into [0, tokens]; an end before its start is an empty
 *            sequence.  They must not fall: results are then unspecified for
 *            all sequences; no access leaves the tensors.
 * All sequences together have at most 2^31 - 513 tokens.
 */
typedef struct ps_linrec_shape {
    int64_t num_seqs;
    int64_t tokens;
    const int32_t *cu_seqlens;
    int64_t channels;
    ps_real type;        /* of x, h and their gradients */
    ps_real gate_type;   /* of g and its gradient: PS_REAL_F32, or `type` */
    int32_t tied;        /* 0: w = 1; otherwise w = 1 - exp(g) */
} ps_linrec_shape;

/*
 * Bytes of workspace of ps_linrec_forward and, with train != 0, of the buffer
 * that a training step's forward call leaves for ps_linrec_backward (0 for
 * shapes that the calls refuse).  256-byte aligned.  Every shape's holds room for
 * a copy of the states, which calls in place (ht == h0, dh0 == d_ht) need.
 */
size_t ps_linrec_workspace_size(const ps_linrec_shape *shape, int train);

/*
 * Forward over whole sequences.
 *   h0  [num_seqs, channels] f32 states at the start, NULL for 0
 *   ht  the same shape, receives the states at the end; may be NULL, or h0
 *       (not in training)
 *   h   contiguous [tokens of all sequences, channels]; tokens that no
 *       sequence holds are left as they are
 *   train != 0: `ws` keeps what ps_linrec_backward reads
 * An empty sequence hands its state on.
 */
ps_status ps_linrec_forward(const ps_linrec_shape *shape, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                            const float *h0, float *ht, void *h, int train, void *ws, size_t ws_bytes,
                            ps_stream_t stream);

/*
 * Backward of one ps_linrec_forward(train != 0) call with the same shape, x,
 * g and h0; `ws` is that call's workspace, which any number of backward calls
 * may use one after the other but which must not change otherwise.
 *   d_h     gradient of h;  d_ht  gradient of ht or NULL (0)
 *   dx, dg  contiguous [tokens of all sequences, channels], of x's and g's type
 *   dh0     gradient of h0, or NULL; may be d_ht
 * Gradients of tokens that no sequence holds are 0.
 */
ps_status ps_linrec_backward(const ps_linrec_shape *shape, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                             const float *h0, const ps_linrec_tensor *d_h, const float *d_ht, void *dx, void *dg,
                             float *dh0, void *ws, size_t ws_bytes, ps_stream_t stream);

/*
 * The recurrence for the next token or few of many sequences, on states that
 * lie in pages of a pool.
 *   tokens    t >= 0 tokens of each sequence (shape->cu_seqlens must be NULL)
 *   state     contiguous [pages, channels] f32, advanced in place
 *   slots     device [num_seqs]: the page of each sequence's state; pages must
 *             differ.  An index outside [0, pages) (-1, say) is a sequence
 *             that takes no part: its outputs are 0.  NULL: page i for i.
 *   lengths   device [num_seqs]: how many of the t tokens count (clamped to
 *             [0, t]); outputs past them are 0.  NULL: all of them.
 *   h         contiguous [num_seqs, t, channels]
 * No workspace.
 */
ps_status ps_linrec_step(const ps_linrec_shape *shape, const ps_linrec_tensor *x, const ps_linrec_tensor *g,
                         float *state, int64_t pages, const int32_t *slots, const int32_t *lengths, void *h,
                         ps_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PREFIX_SCAN_RECURRENCE_H */
